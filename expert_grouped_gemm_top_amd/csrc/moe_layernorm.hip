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
//
// bf16, rows of 4096: forward 16384 rows 55 us, 4.9 TB/s, what a large copy
// reaches; backward 8192 rows 47 us, 4.3 TB/s, and 5 us for the partials (one
// workgroup per row without the prefetch, 512 partial rows: 75 + 7 us).  A wave
// per row of 4096 (no barrier, 128 more registers) was slower: 64 and 66 us.
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
                                                                    float* __restrict__ mean, float* __restrict__ rstd,
                                                                    bool stream) {
  __shared__ float s_sum[2][kWaves];
  const int w = threadIdx.x >> 6;
  const int64_t t = (int64_t)group_id() * (kWaves / WPR) + w / WPR;
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
    store8(y + t * H + c, v[i], stream);
  }
  if (r0 == 0 && mean != nullptr) {
    mean[t] = mu;
    rstd[t] = r;
  }
}

// KW waves per workgroup, KW / WPR rows at a time; the next rows' x and dy are
// loaded under the present ones' sums.  dynamic LDS: 2 H floats.
template <typename T, int WPR, int NC, int KW>
__global__ __launch_bounds__(64 * KW) void layernorm_bwd_kernel(int rows, int H, const T* x,
                                                                const T* __restrict__ gamma,
                                                                const float* __restrict__ mean,
                                                                const float* __restrict__ rstd, const T* dy,
                                                                const T* dx_add, T* dx, float* __restrict__ part,
                                                                bool stream) {
  constexpr int RPW = KW / WPR;
  __shared__ float s_sum[2][KW][2];
  extern __shared__ __attribute__((aligned(16))) float s_col[];
  const int w = threadIdx.x >> 6, slot = w / WPR;
  const int r0 = 8 * ((w % WPR) * 64 + (threadIdx.x & 63));
  Raw8<T> ga[NC], nx[NC], nd[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (r0 + 512 * WPR * i < H) ga[i].load(gamma + r0 + 512 * WPR * i);
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = r0 + 512 * WPR * i;
      if (c < H) {
        nx[i].load(x + t * H + c);
        nd[i].load(dy + t * H + c);
      }
    }
  };
  float dga[NC][8] = {}, dbe[NC][8] = {};
  const float inv = 1.0f / (float)H;
  const int64_t stride = (int64_t)gridDim.x * RPW, first = (int64_t)blockIdx.x * RPW;
  if (first + slot < rows) fetch(first + slot);
  int turn = 0;
  for (int64_t base = first; base < rows; base += stride, turn ^= 1) {
    const int64_t t = base + slot;
    const bool live = t < rows;  // wave-uniform: a slot past the end still meets the others' barriers
    float xh[NC][8], g[NC][8], sg = 0.0f, sgx = 0.0f, r = 0.0f;
    if (live) {
      const float mu = mean[t];
      r = rstd[t];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (r0 + 512 * WPR * i >= H) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = nd[i].get(j);
          xh[i][j] = (nx[i].get(j) - mu) * r;
          dga[i][j] += d * xh[i][j];
          dbe[i][j] += d;
          g[i][j] = d * ga[i].get(j);
          sg += g[i][j];
          sgx += g[i][j] * xh[i][j];
        }
      }
      if (t + stride < rows) fetch(t + stride);
      sg = wave_sum(sg);
      sgx = wave_sum(sgx);
    }
    if constexpr (WPR > 1) {
      // two buffers in turn: a wave may still read the last rows' sums
      if ((threadIdx.x & 63) == 0) {
        s_sum[turn][w][0] = sg;
        s_sum[turn][w][1] = sgx;
      }
      __syncthreads();
      sg = sgx = 0.0f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) {
        sg += s_sum[turn][slot * WPR + i][0];
        sgx += s_sum[turn][slot * WPR + i][1];
      }
    }
    if (!live) continue;
    const float ag = sg * inv, agx = sgx * inv;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = r0 + 512 * WPR * i;
      if (c >= H) continue;
      float add[8] = {};
      if (dx_add != nullptr) load8(dx_add + t * H + c, add);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = r * (g[i][j] - ag - xh[i][j] * agx) + add[j];
      store8(dx + t * H + c, g[i], stream);
    }
  }
  // the slots' column sums meet in LDS in slot order; one partial row each of
  // dgamma and dbeta per workgroup
  for (int q = 0; q < RPW; ++q) {
    if (slot == q) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = r0 + 512 * WPR * i;
        if (c >= H) continue;
        if (q > 0) {
          float u[8], v[8];
          load8(s_col + c, u);
          load8(s_col + H + c, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            dga[i][j] += u[j];
            dbe[i][j] += v[j];
          }
        }
        if (q == RPW - 1) {
          store8(part + (size_t)blockIdx.x * H + c, dga[i]);
          store8(part + ((size_t)gridDim.x + blockIdx.x) * H + c, dbe[i]);
        } else {
          store8(s_col + c, dga[i]);
          store8(s_col + H + c, dbe[i]);
        }
      }
    }
    if (q < RPW - 1) __syncthreads();
  }
}

// out[c] = sum_p part[p][c] in a fixed order: workgroup = 64 columns, wave w
// takes p = w, w + 16, ...; blockIdx.y picks dgamma or dbeta.
template <typename T>
__global__ __launch_bounds__(1024) void column_sum_kernel(int n, int H, const float* __restrict__ part, T* out0,
                                                          T* out1) {
  __shared__ float s[16][64];
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
  const int c = blockIdx.x * 64 + l;
  T* out = blockIdx.y ? out1 : out0;
  if (out == nullptr) return;  // the whole workgroup
  const float* src = part + (size_t)blockIdx.y * n * H;
  float v = 0.0f;
  if (c < H)
#pragma unroll 16
    for (int p = w; p < n; p += 16) v += src[(size_t)p * H + c];
  s[w][l] = v;
  __syncthreads();
  if (w == 0 && c < H) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += s[i][l];
    store1(out + c, v);
  }
}

// Waves per workgroup of the backward: as many as its registers let run.
template <typename T, int NC>
constexpr int bwd_waves() { return NC * (int)sizeof(T) <= 4 ? 16 : (NC * sizeof(T) <= 8 ? 8 : 4); }

// One workgroup per CU (its rows a stride apart), two of the smaller ones where each
// still gets two turns of rows; at most 32 MiB of partials each for dgamma and dbeta.
int bwd_groups(int T, int H, int rpw) {
  const int64_t turns = ((int64_t)T + rpw - 1) / rpw;
  const int64_t groups = std::min<int64_t>(std::max<int64_t>(turns / 2, 256), rpw < 4 ? 512 : 256);
  return (int)std::min<int64_t>({turns, groups, ((int64_t)32 << 20) / (4 * H)});
}

// Outputs above the L2s' 32 MiB leave by streaming stores (bf16, forward /
// backward: 8192 x 4096 28.9 -> 23.7 / 50.1 -> 49.4 us, 16384 x 1024 14.8 ->
// 13.6 / 32.4 -> 27.7 us); smaller ones stay for whoever reads them next.
bool past_caches(int T, int H, size_t esize) { return (int64_t)T * H * (int64_t)esize > ((int64_t)32 << 20); }

template <typename T, int WPR, int NC>
struct Norm {
  static hipError_t fwd(int T_, int H, float eps, const void* x, const void* gamma, const void* beta, void* y,
                        float* mean, float* rstd, hipStream_t stream) {
    constexpr int RPW = kWaves / WPR;
    const int64_t groups = ((int64_t)T_ + RPW - 1) / RPW;
    MOE_LAUNCH((layernorm_fwd_kernel<T, WPR, NC>), wide_grid(groups), dim3(64 * kWaves), 0, stream, T_, H, eps,
               (const T*)x, (const T*)gamma, (const T*)beta, (T*)y, mean, rstd, past_caches(T_, H, sizeof(T)));
    return hipGetLastError();
  }
  static hipError_t bwd(int T_, int H, const void* x, const void* gamma, const float* mean, const float* rstd,
                        const void* dy, const void* dx_add, void* dx, void* dgamma, void* dbeta, float* ws,
                        hipStream_t stream) {
    constexpr int KW = bwd_waves<T, NC>(), RPW = KW / WPR;
    const int groups = bwd_groups(T_, H, RPW);
    const size_t lds = RPW > 1 ? (size_t)2 * H * sizeof(float) : 0;
    auto kern = layernorm_bwd_kernel<T, WPR, NC, KW>;
    static PerDeviceOnce once;
    constexpr size_t most = RPW > 1 ? (size_t)2 * 512 * WPR * NC * sizeof(float) : 0;  // at the widest H of this kernel
    hipError_t err = allow_dynamic_lds(once, (const void*)kern, most);
    if (err != hipSuccess) return err;
    MOE_LAUNCH(kern, dim3(groups), dim3(64 * KW), lds, stream, T_, H, (const T*)x, (const T*)gamma, mean, rstd,
               (const T*)dy, (const T*)dx_add, (T*)dx, ws, past_caches(T_, H, sizeof(T)));
    if ((err = hipGetLastError()) != hipSuccess) return err;
    MOE_LAUNCH((column_sum_kernel<T>), dim3((H + 63) / 64, 2), dim3(1024), 0, stream, groups, H, (const float*)ws,
               (T*)dgamma, (T*)dbeta);
    return hipGetLastError();
  }
  static size_t bytes(int T_, int H) {
    return (size_t)bwd_groups(T_, H, bwd_waves<T, NC>() / WPR) * H * 2 * sizeof(float);
  }
};

// A wave per row up to 1024 columns, a workgroup per row above.
constexpr int kWaveRowMax = 1024;

template <typename T, typename Fn>
auto with_norm(int H, Fn&& f) {
  if (H <= 512) return f(Norm<T, 1, 1>{});
  if (H <= kWaveRowMax) return f(Norm<T, 1, 2>{});
  if (H <= 2048) return f(Norm<T, 4, 1>{});
  if (H <= 4096) return f(Norm<T, 4, 2>{});
  if (H <= 8192) return f(Norm<T, 4, 4>{});
  return f(Norm<T, 4, 8>{});
}

}  // namespace

size_t layernorm_workspace_bytes(int T, int H) {
  auto bytes = [&](auto norm) { return norm.bytes(T, H); };
  return std::max(with_norm<float>(H, bytes), with_norm<uint16_t>(H, bytes));
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
