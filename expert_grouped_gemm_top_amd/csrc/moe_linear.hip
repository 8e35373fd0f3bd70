// moe_linear.hip -- dense product with bias, activation, gate and residual in
// its epilogue, and its backward.
//
//   z = x W + bias,  y = act(z) [* mul] [+ residual]
//   dz = dy [* mul] act'(z),  dmul = dy act(z),
//   dx = dz W^T [+ dx_add],  dW = x^T dz,  dbias = sum_t dz
#include <algorithm>
#include <type_traits>

#include "moe_common.h"
#include "moe_launch.h"
#include "moe_rows.h"

namespace moe {

namespace {

enum Act { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

constexpr float kTanhA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

// 1 / (1 + exp(-v))
__device__ __forceinline__ float logistic(float v) { return 1.0f / (1.0f + expf(-v)); }

// act(z); NaN stays NaN.
__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;
    case kActGelu: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    case kActGeluTanh: return z * logistic(2.0f * kTanhA * (z + kTanhB * z * z * z));  // (1 + tanh u) / 2 = logistic(2 u)
    case kActSilu: return z * logistic(z);
    default: return z;
  }
}

// act(z) and act'(z).  The slopes are 0 or 1 to fp32 precision beyond |z| = 30
// (SILU: 100), where their formulas would form 0 * inf.
__device__ __forceinline__ void act_both(int act, float z, float& value, float& slope) {
  switch (act) {
    case kActRelu:
      value = z < 0.0f ? 0.0f : z;
      slope = z > 0.0f ? 1.0f : 0.0f;
      return;
    case kActGelu: {
      const float c = z > 30.0f ? 30.0f : (z < -30.0f ? -30.0f : z);
      const float phi = 0.5f * erfcf(-0.70710678118654752f * c);
      value = z * phi;
      slope = phi + c * 0.3989422804014327f * expf(-0.5f * c * c);
      return;
    }
    case kActGeluTanh: {
      const float c = z > 30.0f ? 30.0f : (z < -30.0f ? -30.0f : z);
      const float s = logistic(2.0f * kTanhA * (c + kTanhB * c * c * c));
      value = z * s;
      slope = s + c * s * (1.0f - s) * 2.0f * kTanhA * (1.0f + 3.0f * kTanhB * c * c);
      return;
    }
    case kActSilu: {
      const float c = z > 100.0f ? 100.0f : (z < -100.0f ? -100.0f : z);
      const float s = logistic(c);
      value = z * s;
      slope = s * (1.0f + c * (1.0f - s));
      return;
    }
    default:
      value = z;
      slope = 1.0f;
  }
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf2f(*p); }

// C [M, N] = A B over K, then the epilogue.  A(m, k) = a[m sam + k sak], B(k, n) = b[k sbk + n sbn].
struct LinearProduct {
  int M, N, K;
  const void* a;
  int64_t sam, sak;
  const void* b;
  int64_t sbk, sbn;
  int act;
  const void *bias, *mul, *residual;
  void *z, *out;
};

// 64 x 64 outputs per workgroup, 4 x 4 per thread, 16 k per stage.
template <typename T>
__global__ __launch_bounds__(256) void linear_product_kernel(LinearProduct g) {
  __shared__ float s_a[16][65], s_b[16][65];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int m0 = blockIdx.x * 64, n0 = blockIdx.y * 64;
  const T* a = (const T*)g.a;
  const T* b = (const T*)g.b;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < g.K; k0 += 16) {
    for (int q = tid; q < 64 * 16; q += 256) {
      const int am = g.sak == 1 ? q >> 4 : q & 63, ak = g.sak == 1 ? q & 15 : q >> 6;
      s_a[ak][am] = m0 + am < g.M && k0 + ak < g.K ? load1(a + (m0 + am) * g.sam + (k0 + ak) * g.sak) : 0.0f;
      const int bn = g.sbk == 1 ? q >> 4 : q & 63, bk = g.sbk == 1 ? q & 15 : q >> 6;
      s_b[bk][bn] = n0 + bn < g.N && k0 + bk < g.K ? load1(b + (k0 + bk) * g.sbk + (n0 + bn) * g.sbn) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(s_a[k][ty + 16 * i], s_b[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= g.M || n >= g.N) continue;
      const size_t at = (size_t)m * g.N + n;
      float z = acc[i][j];
      if (g.bias != nullptr) z += load1((const T*)g.bias + n);
      float y = act_value(g.act, z);
      if (g.mul != nullptr) y *= load1((const T*)g.mul + at);
      if (g.residual != nullptr) y += load1((const T*)g.residual + at);
      if (g.z != nullptr) store1((T*)g.z + at, z);
      store1((T*)g.out + at, y);
    }
}

// dz, dmul and the column sums of dz.  Workgroup = 32 runs of eight columns x 8
// rows at a time, blockIdx.y strides over the rows; each thread keeps its
// columns' sums, the eight of a column meet in LDS and leave one partial row.
template <typename T>
__global__ __launch_bounds__(256) void linear_dz_kernel(int rows, int O, int act, const T* z, const T* mul, const T* dy,
                                                        T* dz, T* dmul, float* __restrict__ part) {
  __shared__ float s_sum[8][32][8];
  const int run = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int c = 8 * (blockIdx.x * 32 + run);
  float sum[8] = {};
  if (c < O) {
    for (int64_t t = (int64_t)blockIdx.y * 8 + sub; t < rows; t += (int64_t)gridDim.y * 8) {
      const size_t at = (size_t)t * O + c;
      float d[8];
      load8(dy + at, d);
      if (z != nullptr) {
        float zv[8], mv[8], dm[8];
        load8(z + at, zv);
        if (mul != nullptr) load8(mul + at, mv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float value, slope;
          act_both(act, zv[j], value, slope);
          dm[j] = d[j] * value;
          d[j] = (mul != nullptr ? d[j] * mv[j] : d[j]) * slope;
        }
        if (mul != nullptr) store8(dmul + at, dm);
        store8(dz + at, d);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += d[j];
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) s_sum[sub][run][j] = sum[j];
  __syncthreads();
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col >= O) return;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v += s_sum[i][threadIdx.x >> 3][threadIdx.x & 7];
  part[(size_t)blockIdx.y * O + col] = v;
}

// out[c] = sum_p part[p][c], p ascending within each of four waves, then the waves.
template <typename T>
__global__ __launch_bounds__(256) void linear_dbias_kernel(int n, int O, const float* __restrict__ part, T* out) {
  __shared__ float s[4][64];
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63, c = blockIdx.x * 64 + l;
  float v = 0.0f;
  if (c < O)
    for (int p = w; p < n; p += 4) v += part[(size_t)p * O + c];
  s[w][l] = v;
  __syncthreads();
  if (w == 0 && c < O) store1(out + c, s[0][l] + s[1][l] + s[2][l] + s[3][l]);
}

// Row slots of linear_dz_kernel: about 1024 workgroups, eight rows each at least.
int dz_slots(int T, int O) {
  const int cols = (O + 255) / 256;
  return std::max(1, std::min((T + 7) / 8, 1024 / std::min(cols, 1024)));
}

template <typename T>
hipError_t product(const LinearProduct& g, hipStream_t stream) {
  MOE_LAUNCH((linear_product_kernel<T>), dim3((g.M + 63) / 64, (g.N + 63) / 64), dim3(256), 0, stream, g);
  return hipGetLastError();
}

template <typename T>
hipError_t linear_bwd_typed(const LinearArgs& g, const void* z, const void* mul, const void* dy, void* dz,
                            const void* dx_add, void* dx, void* dw, void* dbias, void* dmul, float* ws,
                            hipStream_t stream) {
  const bool plain = g.act == kActNone && mul == nullptr;
  const int T_ = g.T, I = g.I, O = g.O;
  if (!plain || dbias != nullptr) {
    const int slots = dz_slots(T_, O);
    MOE_LAUNCH((linear_dz_kernel<T>), dim3((O + 255) / 256, slots), dim3(256), 0, stream, T_, O, g.act,
               plain ? nullptr : (const T*)z, (const T*)mul, (const T*)dy, (T*)dz, (T*)dmul,
               dbias != nullptr ? ws : nullptr);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (dbias != nullptr) {
      MOE_LAUNCH((linear_dbias_kernel<T>), dim3((O + 63) / 64), dim3(256), 0, stream, slots, O, (const float*)ws,
                 (T*)dbias);
      if ((err = hipGetLastError()) != hipSuccess) return err;
    }
  }
  const void* d = plain ? dy : dz;
  if (dx != nullptr) {
    LinearProduct p{T_, I, O, d, O, 1, g.w, 1, O, kActNone, nullptr, nullptr, dx_add, nullptr, dx};
    hipError_t err = product<T>(p, stream);
    if (err != hipSuccess) return err;
  }
  if (dw != nullptr) {
    LinearProduct p{I, O, T_, g.x, 1, I, d, O, 1, kActNone, nullptr, nullptr, nullptr, nullptr, dw};
    return product<T>(p, stream);
  }
  return hipSuccess;
}

}  // namespace

size_t linear_workspace_bytes(int T, int I, int O, int esize) {
  (void)I;
  (void)esize;
  return (size_t)dz_slots(T, O) * O * sizeof(float);
}

hipError_t launch_linear_fwd(const LinearArgs& g, int esize, const void* bias, const void* mul, const void* residual,
                             void* z, void* y, void* ws, hipStream_t stream) {
  (void)ws;
  const LinearProduct p{g.T, g.O, g.I, g.x, g.I, 1, g.w, g.O, 1, g.act, bias, mul, residual, z, y};
  return esize == 4 ? product<float>(p, stream) : product<uint16_t>(p, stream);
}

hipError_t launch_linear_bwd(const LinearArgs& g, int esize, const void* z, const void* mul, const void* dy, void* dz,
                             const void* dx_add, void* dx, void* dw, void* dbias, void* dmul, void* ws,
                             hipStream_t stream) {
  return esize == 4 ? linear_bwd_typed<float>(g, z, mul, dy, dz, dx_add, dx, dw, dbias, dmul, (float*)ws, stream)
                    : linear_bwd_typed<uint16_t>(g, z, mul, dy, dz, dx_add, dx, dw, dbias, dmul, (float*)ws, stream);
}

}  // namespace moe
