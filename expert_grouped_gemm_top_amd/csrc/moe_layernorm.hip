// moe_layernorm.hip -- layer norm over rows, forward and backward.
//
//   y = (x - mean) rstd gamma + beta,  rstd = 1 / sqrt(var + eps)
//   dx = rstd (g - avg(g) - xh avg(g xh)) [+ dx_add],  g = dy gamma,  xh = (x - mean) rstd
//   dgamma = sum_t dy xh,  dbeta = sum_t dy
//
// HBM-bound: a row is read once and held in registers, by WPR waves with NC
// runs of eight elements per lane; all sums fp32, the variance from the
// differences to the mean.  The backward's workgroups walk the rows with a
// fixed stride and keep their columns' dgamma and dbeta in registers; each
// leaves one partial row, and a second kernel adds those in order (no atomics,
// so the result does not depend on the schedule).
#include <algorithm>

#include "moe_common.h"
#include "moe_launch.h"
#include "moe_rows.h"

namespace moe {

namespace {

constexpr int kWaves = 4;  // per workgroup

// Sum over the WPR waves that share a row; `s` holds one float per wave and
// call site.  Every wave of the workgroup calls it the same number of times.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* s) {
  v = wave_sum(v);
  if constexpr (WPR > 1) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) s[w] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) v += s[(w / WPR) * WPR + i];
  }
  return v;
}

template <typename T, int WPR, int NC>
__global__ __launch_bounds__(64 * kWaves) void layernorm_fwd_kernel(int rows, int H, float eps,
                                                                    const T* x, const T* __restrict__ gamma,
                                                                    const T* __restrict__ beta, T* y,
                                                                    float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float s_sum[2][kWaves];
  const int w = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * (kWaves / WPR) + w / WPR;
  const bool live = t < rows;
  const int r0 = 8 * ((w % WPR) * 64 + (threadIdx.x & 63));  // first column of this lane's runs
  const T* xr = x + (live ? t : 0) * H;
  float v[NC][8], sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = r0 + 512 * WPR * i;
    if (c < H) {
      load8(xr + c, v[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += v[i][j];
    }
  }
  const float mu = row_sum<WPR>(sum, s_sum[0]) / (float)H;
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (r0 + 512 * WPR * i < H)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] -= mu;
        sq += v[i][j] * v[i][j];
      }
  const float r = 1.0f / sqrtf(row_sum<WPR>(sq, s_sum[1]) / (float)H + eps);
  if (!live) return;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = r0 + 512 * WPR * i;
    if (c >= H) continue;
    float ga[8], be[8];
    load8(gamma + c, ga);
    if (beta != nullptr) load8(beta + c, be);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float n = v[i][j] * r;
      v[i][j] = beta != nullptr ? n * ga[j] + be[j] : n * ga[j];
    }
    store8(y + t * H + c, v[i]);
  }
  if (r0 == 0 && mean != nullptr) {
    mean[t] = mu;
    rstd[t] = r;
  }
}

template <typename T, int WPR, int NC>
__global__ __launch_bounds__(64 * kWaves) void layernorm_bwd_kernel(int rows, int H, const T* __restrict__ x,
                                                                    const T* __restrict__ gamma,
                                                                    const float* __restrict__ mean,
                                                                    const float* __restrict__ rstd, const T* dy,
                                                                    const T* dx_add, T* dx, float* __restrict__ part) {
  __shared__ float s_sum[2][2][kWaves];
  constexpr int RPW = kWaves / WPR;  // rows of a workgroup at a time
  const int w = threadIdx.x >> 6;
  const int r0 = 8 * ((w % WPR) * 64 + (threadIdx.x & 63));
  float dga[NC][8] = {}, dbe[NC][8] = {};
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * RPW; base < rows; base += (int64_t)gridDim.x * RPW, turn ^= 1) {
    const int64_t t = base + w / WPR;
    const bool live = t < rows;
    const int64_t at = (live ? t : base) * H;
    const float mu = mean[live ? t : base], r = rstd[live ? t : base];
    float xh[NC][8], g[NC][8], sg = 0.0f, sgx = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = r0 + 512 * WPR * i;
      if (c >= H) continue;
      float ga[8];
      load8(x + at + c, xh[i]);
      load8(dy + at + c, g[i]);
      load8(gamma + c, ga);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] = (xh[i][j] - mu) * r;
        const float d = live ? g[i][j] : 0.0f;
        dga[i][j] += d * xh[i][j];
        dbe[i][j] += d;
        g[i][j] = d * ga[j];
        sg += g[i][j];
        sgx += g[i][j] * xh[i][j];
      }
    }
    // two buffers in turn: a wave may still read the last row's sums
    const float ag = row_sum<WPR>(sg, s_sum[turn][0]) / (float)H;
    const float agx = row_sum<WPR>(sgx, s_sum[turn][1]) / (float)H;
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = r0 + 512 * WPR * i;
      if (c >= H) continue;
      float add[8] = {};
      if (dx_add != nullptr) load8(dx_add + at + c, add);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = r * (g[i][j] - ag - xh[i][j] * agx) + add[j];
      store8(dx + at + c, g[i]);
    }
  }
  // partial rows: part[0][p], part[1][p] for p = the workgroup's row slot
  const size_t slots = (size_t)gridDim.x * RPW, p = (size_t)blockIdx.x * RPW + w / WPR;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = r0 + 512 * WPR * i;
    if (c >= H) continue;
    store8(part + p * H + c, dga[i]);
    store8(part + (slots + p) * H + c, dbe[i]);
  }
}

// out[c] = sum_p part[p][c] in a fixed order: workgroup = 64 columns, wave w
// takes p = w, w + 4, ...; blockIdx.y picks dgamma or dbeta.
template <typename T>
__global__ __launch_bounds__(256) void column_sum_kernel(int n, int H, const float* __restrict__ part, T* out0,
                                                         T* out1) {
  __shared__ float s[4][64];
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
  const int c = blockIdx.x * 64 + l;
  T* out = blockIdx.y ? out1 : out0;
  if (out == nullptr) return;  // the whole workgroup
  const float* src = part + (size_t)blockIdx.y * n * H;
  float v = 0.0f;
  if (c < H)
#pragma unroll 8
    for (int p = w; p < n; p += 4) v += src[(size_t)p * H + c];
  s[w][l] = v;
  __syncthreads();
  if (w == 0 && c < H) store1(out + c, s[0][l] + s[1][l] + s[2][l] + s[3][l]);
}

// Partial rows of the backward: enough workgroups to fill the chip, at most 32 MiB of them each for dgamma and dbeta.
int bwd_groups(int T, int H, int rpw) {
  const int64_t want = std::min<int64_t>((T + rpw - 1) / rpw, 512);
  const int64_t fit = std::max<int64_t>(1, ((int64_t)32 << 20) / ((int64_t)4 * H * rpw));
  return (int)std::min(want, fit);
}

template <typename T, int WPR, int NC>
struct Norm {
  static hipError_t fwd(int T_, int H, float eps, const void* x, const void* gamma, const void* beta, void* y,
                        float* mean, float* rstd, hipStream_t stream) {
    constexpr int RPW = kWaves / WPR;
    MOE_LAUNCH((layernorm_fwd_kernel<T, WPR, NC>), dim3((T_ + RPW - 1) / RPW), dim3(64 * kWaves), 0, stream, T_, H,
               eps, (const T*)x, (const T*)gamma, (const T*)beta, (T*)y, mean, rstd);
    return hipGetLastError();
  }
  static hipError_t bwd(int T_, int H, const void* x, const void* gamma, const float* mean, const float* rstd,
                        const void* dy, const void* dx_add, void* dx, void* dgamma, void* dbeta, float* ws,
                        hipStream_t stream) {
    constexpr int RPW = kWaves / WPR;
    const int groups = bwd_groups(T_, H, RPW);
    MOE_LAUNCH((layernorm_bwd_kernel<T, WPR, NC>), dim3(groups), dim3(64 * kWaves), 0, stream, T_, H, (const T*)x,
               (const T*)gamma, mean, rstd, (const T*)dy, (const T*)dx_add, (T*)dx, ws);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    MOE_LAUNCH((column_sum_kernel<T>), dim3((H + 63) / 64, 2), dim3(256), 0, stream, groups * RPW, H,
               (const float*)ws, (T*)dgamma, (T*)dbeta);
    return hipGetLastError();
  }
};

// A wave per row up to 1024 columns, a workgroup per row above.
constexpr int kWaveRowMax = 1024;

template <typename T, typename Fn>
hipError_t with_norm(int H, Fn&& f) {
  if (H <= 512) return f(Norm<T, 1, 1>{});
  if (H <= kWaveRowMax) return f(Norm<T, 1, 2>{});
  if (H <= 2048) return f(Norm<T, 4, 1>{});
  if (H <= 4096) return f(Norm<T, 4, 2>{});
  if (H <= 8192) return f(Norm<T, 4, 4>{});
  return f(Norm<T, 4, 8>{});
}

}  // namespace

size_t layernorm_workspace_bytes(int T, int H) {
  const int rpw = H <= kWaveRowMax ? kWaves : 1;
  return (size_t)bwd_groups(T, H, rpw) * rpw * H * 2 * sizeof(float);
}

hipError_t launch_layernorm_fwd(int T, int H, int esize, float eps, const void* x, const void* gamma, const void* beta,
                                void* y, float* mean, float* rstd, hipStream_t stream) {
  auto run = [&](auto norm) { return norm.fwd(T, H, eps, x, gamma, beta, y, mean, rstd, stream); };
  return esize == 4 ? with_norm<float>(H, run) : with_norm<uint16_t>(H, run);
}

hipError_t launch_layernorm_bwd(int T, int H, int esize, const void* x, const void* gamma, const float* mean,
                                const float* rstd, const void* dy, const void* dx_add, void* dx, void* dgamma,
                                void* dbeta, void* ws, hipStream_t stream) {
  auto run = [&](auto norm) {
    return norm.bwd(T, H, x, gamma, mean, rstd, dy, dx_add, dx, dgamma, dbeta, (float*)ws, stream);
  };
  return esize == 4 ? with_norm<float>(H, run) : with_norm<uint16_t>(H, run);
}

}  // namespace moe
