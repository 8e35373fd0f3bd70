// moe_linear.hip -- dense product with bias, activation, gate and residual in
// its epilogue, and its backward.
//
//   z = x W + bias,  y = act(z) [* mul] [+ residual]
//   dz = dy [* mul] act'(z),  dmul = dy act(z),
//   dx = dz W^T [+ dx_add],  dW = x^T dz,  dbias = sum_t dz
//
// The products run on the matrix cores from LDS tiles: bf16 on 32x32x16, fp32 on
// 32x32x2.  Sums are fp32 throughout.  The backward rounds dz to the element
// type once, as the operand of both products and a tensor the caller keeps:
// that adds an error as large as the outputs' own rounding (2^-9 of dx and dW
// in the root mean square); dbias sums the unrounded values.
#include <algorithm>

#include "moe_common.h"
#include "moe_launch.h"
#include "moe_linear_plan.h"
#include "moe_rows.h"
#include "moe_tile.h"

namespace moe {

namespace {

enum Act { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

constexpr float kTanhA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

// Logistic function and normal distribution of an activation, by the element type.
// bf16: on the hardware's exp2 (quick_exp) and reciprocal, the distribution
// within 1.5e-7 (5e-5 of itself at -3, 2^-9 from -5.2 on, where it is below
// 1e-7): the library's expf, erfcf and division took 7 of 28 us of a GELU
// product's epilogue at 4099 x 768.  fp32: those, whose errors are a few 2^-24
// of the result in the tails too; they cost its products 0.2 to 0.7 us
// (4096 x 512 -> 1024 with GELU and a gate 45.5 us).
template <typename T>
__device__ __forceinline__ float exp_of(float v) {
  return sizeof(T) == 4 ? expf(v) : quick_exp(v);
}

// s = 1 / (1 + exp(-v)), and `rest` = 1 - s.
struct Logistic {
  float s, rest;
};
template <typename T>
__device__ __forceinline__ Logistic logistic(float v) {
  if constexpr (sizeof(T) == 2) {
    const float s = __builtin_amdgcn_rcpf(1.0f + quick_exp(-v));
    return {s, 1.0f - s};
  } else {
    const float e = expf(-fabsf(v)), near = 1.0f / (1.0f + e), far = e / (1.0f + e);
    return v >= 0.0f ? Logistic{near, far} : Logistic{far, near};
  }
}

// Phi(z), the normal distribution: erfc(-z / sqrt 2) / 2.  bf16: by formula
// 7.1.26 of Abramowitz and Stegun, erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2),
// t = 1 / (1 + p x), |error| <= 1.5e-7, mirrored for z > 0.
template <typename T>
__device__ __forceinline__ float normal_cdf(float z) {
  if constexpr (sizeof(T) == 4) return 0.5f * erfcf(-z * 0.70710678f);
  const float x = fabsf(z) * 0.70710678f;
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * x);
  const float poly =
      t * (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
  const float tail = 0.5f * poly * quick_exp(-x * x);
  return z > 0.0f ? 1.0f - tail : tail;
}

// v = act(v) for eight values of an output of type T; NaN stays NaN.  One branch per run, not per value.
template <typename T>
__device__ __forceinline__ void act8(int act, float (&v)[8]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];
      return;
    case kActGelu:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= normal_cdf<T>(v[j]);
      return;
    case kActGeluTanh:  // (1 + tanh u) / 2 = logistic(2 u)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= logistic<T>(2.0f * kTanhA * (v[j] + kTanhB * v[j] * v[j] * v[j])).s;
      return;
    case kActSilu:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= logistic<T>(v[j]).s;
      return;
    default: return;
  }
}

__device__ __forceinline__ float clamped(float z, float most) { return z > most ? most : (z < -most ? -most : z); }

// value = act(z) and slope = act'(z) for eight values.  Slopes, and the factor of z
// in the values, are 0 or 1 in fp32 beyond |z| = 30 (SILU: 110, exp(-110) is below
// the smallest subnormal), where the slopes' formulas would form 0 * inf.
template <typename T>
__device__ __forceinline__ void act8_both(int act, const float (&z)[8], float (&value)[8], float (&slope)[8]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        value[j] = z[j] < 0.0f ? 0.0f : z[j];
        slope[j] = z[j] > 0.0f ? 1.0f : 0.0f;
      }
      return;
    case kActGelu:
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float c = clamped(z[j], 30.0f), phi = normal_cdf<T>(c);
        value[j] = z[j] * phi;
        slope[j] = phi + c * 0.3989422804014327f * exp_of<T>(-0.5f * c * c);
      }
      return;
    case kActGeluTanh:
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float c = clamped(z[j], 30.0f);
        const Logistic u = logistic<T>(2.0f * kTanhA * (c + kTanhB * c * c * c));
        value[j] = z[j] * u.s;
        slope[j] = u.s + c * u.s * u.rest * 2.0f * kTanhA * (1.0f + 3.0f * kTanhB * c * c);
      }
      return;
    case kActSilu:
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float c = clamped(z[j], 110.0f);
        const Logistic u = logistic<T>(c);
        value[j] = z[j] * u.s;
        slope[j] = u.s * (1.0f + c * u.rest);
      }
      return;
    default:
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        value[j] = z[j];
        slope[j] = 1.0f;
      }
  }
}

// C [M, N] = A B over K, then the epilogue.
struct LinearProduct : TileSource {
  int K;
  int act;
  const void *bias, *mul, *residual;
  void *z, *out;
  int slice;    // k per slice of a split reduction, a multiple of 128 (>= K: not split)
  float* part;  // split: fp32 partials [slices][M][N]
};

// The epilogue of eight neighbouring outputs, from their fp32 sums.
template <typename T>
__device__ __forceinline__ void finish8(const LinearProduct& g, int64_t m, int n, float (&v)[8]) {
  const int64_t at = m * g.N + n;
  float u[8];
  if (g.bias != nullptr) {
    load8((const T*)g.bias + n, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += u[j];
  }
  if (g.z != nullptr) store8((T*)g.z + at, v);
  act8<T>(g.act, v);
  if (g.mul != nullptr) {
    load8((const T*)g.mul + at, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= u[j];
  }
  if (g.residual != nullptr) {
    load8((const T*)g.residual + at, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += u[j];
  }
  store8((T*)g.out + at, v);
}

// Eight outputs of a tile: to the slice's partials or through the epilogue.
template <typename T>
struct Leave {
  template <typename C>
  static constexpr bool kWhole = false;
  const LinearProduct& g;
  int slice;
  // N is a multiple of 8: a run is all in or all out
  __device__ __forceinline__ bool skip(int m, int n) const { return m >= g.M || n >= g.N; }
  template <typename Lanes>
  __device__ __forceinline__ void operator()(int64_t m, int n, float (&v)[8], Lanes) const {
    if (g.part != nullptr) store8(g.part + ((int64_t)slice * g.M + m) * g.N + n, v);
    else finish8<T>(g, m, n, v);
  }
};

// Adds the slices of split reductions in order, then the epilogue: `first`
// workgroups for one product, the others for a second one.
template <typename T>
__global__ __launch_bounds__(256) void linear_slices_kernel(LinearProduct g0, LinearProduct g1, int first) {
  const bool second = (int)blockIdx.x >= first;
  const LinearProduct& g = second ? g1 : g0;
  const int groups = second ? gridDim.x - first : first, group = second ? blockIdx.x - first : blockIdx.x;
  const int runs = g.N / 8, slices = (g.K + g.slice - 1) / g.slice;
  const int64_t total = (int64_t)g.M * runs, MN = (int64_t)g.M * g.N;
  for (int64_t i = (int64_t)group * 256 + threadIdx.x; i < total; i += (int64_t)groups * 256) {
    float v[8], u[8];
    load8(g.part + 8 * i, v);
    for (int s = 1; s < slices; ++s) {
      load8(g.part + s * MN + 8 * i, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += u[j];
    }
    finish8<T>(g, i / runs, 8 * (int)(i % runs), v);
  }
}

template <typename T, bool AKC, bool BKC, typename C, bool TAIL>
__device__ __forceinline__ void any_product(const LinearProduct& g, int item, unsigned char* s_dyn) {
  const int mtiles = (g.M + C::BM - 1) / C::BM, ntiles = (g.N + C::BN - 1) / C::BN, tiles = mtiles * ntiles;
  const int slice = item / tiles;
  if (slice * (int64_t)g.slice >= g.K) return;  // past the last slice: the grid may hold a few more
  int mt, nt;
  tile_of(item % tiles, mtiles, ntiles, 1024 / C::BM, mt, nt);
  const int kb = slice * g.slice;
  tile_product<T, AKC, BKC, C, TAIL>(g, mt, nt, kb, min(g.K, kb + g.slice), s_dyn, Leave<T>{g, slice});
}

// One workgroup per tile and slice: x W.
template <typename T, typename C, bool TAIL>
__global__ __launch_bounds__(kTileThreads, 2) void linear_fwd_kernel(LinearProduct g) {
  extern __shared__ __attribute__((aligned(16))) unsigned char s_dyn[];
  any_product<T, true, false, C, TAIL>(g, group_id(), s_dyn);
}

// The backward's products in one launch, so that one's workgroups fill the CUs
// that the other leaves idle: `nw` workgroups of x^T dz, `nx` of dz W^T (the
// longer ones first), and behind them the sums of dbias' partial rows.  Both
// products at 4099 x 2048 x 768: 46 us, in launches of their own 30 + 30; at
// 128 x 2048 x 768 8.1 us, 8.0 + 8.4; at 8192 x 4096 x 1408 220 us (0.86
// PFLOP/s), on operands of zeros 194 us: a ninth of it goes with the power that
// the values' switching draws.
struct ColumnSum {
  const float* part;
  int n, cols;
  void* out;
};

template <typename T>
__device__ __forceinline__ void column_sum(const ColumnSum& c, int block, float* s) {
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63, col = block * 64 + l;
  if (c.out == nullptr) return;
  float v = 0.0f;
  if (col < c.cols)
#pragma unroll 8
    for (int p = w; p < c.n; p += kTileThreads / 64) v += c.part[(size_t)p * c.cols + col];
  s[w * 64 + l] = v;
  __syncthreads();
  if (w != 0 || col >= c.cols) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < kTileThreads / 64; ++i) v += s[i * 64 + l];
  store1((T*)c.out + col, v);
}

template <typename T, typename CX, typename CW, bool TAIL>
__global__ __launch_bounds__(kTileThreads, 2) void linear_bwd_kernel(LinearProduct gx, LinearProduct gw, ColumnSum sum,
                                                                 int nx, int nw, int x_first) {
  extern __shared__ __attribute__((aligned(16))) unsigned char s_dyn[];
  const int b = group_id();
  if (b >= nx + nw) return column_sum<T>(sum, b - nx - nw, reinterpret_cast<float*>(s_dyn));
  const bool is_x = x_first ? b < nx : b >= nw;
  if (is_x) any_product<T, true, true, CX, TAIL>(gx, x_first ? b : b - nw, s_dyn);
  else any_product<T, false, false, CW, TAIL>(gw, x_first ? b - nx : b, s_dyn);
}

// dz, dmul and the column sums of dz.  HBM-bound: 25 us at 8192 x 1408 with a
// gate (three tensors read, two written, 4.6 TB/s).  Workgroup = 32 runs of eight columns x 8
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
        float zv[8], value[8], slope[8];
        load8(z + at, zv);
        act8_both<T>(act, zv, value, slope);
        if (mul != nullptr) {
          float mv[8];
          load8(mul + at, mv);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            value[j] *= d[j];
            d[j] *= mv[j];
          }
          store8(dmul + at, value);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] *= slope[j];
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

// Row slots of linear_dz_kernel: about 1024 workgroups, eight rows each at least.
int dz_slots(int T, int O) {
  const int cols = (O + 255) / 256;
  return std::max(1, std::min((T + 7) / 8, 1024 / std::min(cols, 1024)));
}
size_t dbias_bytes(int T, int O) { return ((size_t)dz_slots(T, O) * O * sizeof(float) + 15) / 16 * 16; }

// ---- launchers -------------------------------------------------------------------

const Cut& fwd_cut(int T, int I, int O, int esize) {
  return remembered<Cut>(T, I, O, esize, [&] { return plan_fwd(T, O, I, esize); });
}
const Plan2& bwd_cuts(int T, int I, int O, int esize, bool dx, bool dw) {
  return remembered<Plan2>(T, I, O, esize + (dx ? 8 : 0) + (dw ? 16 : 0),
                           [&] { return plan_bwd(T, I, O, esize, dx, dw); });
}

size_t slice_bytes(int M, int N, const Cut& c) {
  return c.slices > 1 ? ((size_t)c.slices * M * N * sizeof(float) + 15) / 16 * 16 : 0;
}

// The sums of up to two split products (those with partials) in one launch.
template <typename T>
hipError_t add_slices(const LinearProduct& a, const LinearProduct& b, hipStream_t stream) {
  auto groups = [](const LinearProduct& g) {
    const int64_t runs = (int64_t)g.M * (g.N / 8);
    return g.part == nullptr ? 0 : (int)std::min<int64_t>((runs + 255) / 256, 2048);
  };
  const int ga = groups(a), gb = groups(b);
  if (ga + gb == 0) return hipSuccess;
  MOE_LAUNCH((linear_slices_kernel<T>), dim3(ga + gb), dim3(256), 0, stream, a, b, ga);
  return hipGetLastError();
}

// Whether stages of C reach past the product's edges and must be masked: every
// stage of every slice is whole where this is false (one that ran past the
// reduction's end would read past the operands).
template <typename T, bool AKC, bool BKC, typename C>
bool has_tail(const LinearProduct& g) {
  constexpr int STAGE_K = kStageK<T> * C::KG;
  return g.K % STAGE_K != 0 || g.slice % STAGE_K != 0 || (!BKC && g.N % C::BN != 0) ||
         (!AKC && g.M % C::BM != 0);
}

template <typename T, typename C, bool TAIL>
hipError_t run_fwd(const LinearProduct& g, int64_t groups, hipStream_t stream) {
  auto kern = linear_fwd_kernel<T, C, TAIL>;
  static PerDeviceOnce once;
  hipError_t err = allow_dynamic_lds(once, (const void*)kern, C::LDS);
  if (err != hipSuccess) return err;
  MOE_LAUNCH(kern, wide_grid(groups), dim3(kTileThreads), C::LDS, stream, g);
  return hipGetLastError();
}

template <typename T>
hipError_t linear_fwd_typed(LinearProduct g, float* ws, hipStream_t stream) {
  const Cut& c = fwd_cut(g.M, g.K, g.N, sizeof(T));
  g.slice = c.slice;
  g.part = c.slices > 1 ? ws : nullptr;
  auto run = [&](auto tile) {
    using C = decltype(tile);
    return has_tail<T, true, false, C>(g) ? run_fwd<T, C, true>(g, c.groups, stream)
                                          : run_fwd<T, C, false>(g, c.groups, stream);
  };
  hipError_t err = hipErrorUnknown;
  if constexpr (sizeof(T) == 2) {
    if (c.tile == kTile256x256) err = run(Tile0{});
    if (c.tile == kTile256x128) err = run(Tile1{});
  }
  if (c.tile == kTile128x128) err = run(Tile2{});
  if (c.tile == kTile128x64) err = run(Tile3{});
  if (c.tile == kTile64x64) err = run(Tile4<T>{});
  if (c.tile == kTile32x32) err = run(Tile5{});
  if (err != hipSuccess) return err;
  return add_slices<T>(g, LinearProduct{}, stream);
}

template <typename T, typename CX, typename CW, bool TAIL>
hipError_t run_bwd(const LinearProduct& gx, const LinearProduct& gw, const ColumnSum& sum, const Plan2& p,
                   hipStream_t stream) {
  constexpr size_t lds = std::max(CX::LDS, CW::LDS);
  auto kern = linear_bwd_kernel<T, CX, CW, TAIL>;
  static PerDeviceOnce once;
  hipError_t err = allow_dynamic_lds(once, (const void*)kern, lds);
  if (err != hipSuccess) return err;
  const int64_t sums = sum.out != nullptr ? (sum.cols + 63) / 64 : 0;
  MOE_LAUNCH(kern, wide_grid(p.x.groups + p.w.groups + sums), dim3(kTileThreads), lds, stream, gx, gw, sum,
             (int)p.x.groups, (int)p.w.groups, p.x.each > p.w.each ? 1 : 0);
  return hipGetLastError();
}

template <typename T>
hipError_t linear_bwd_typed(const LinearArgs& g, const void* z, const void* mul, const void* dy, void* dz,
                            const void* dx_add, void* dx, void* dw, void* dbias, void* dmul, float* ws,
                            hipStream_t stream) {
  const bool plain = g.act == kActNone && mul == nullptr;
  const int T_ = g.T, I = g.I, O = g.O, slots = dz_slots(T_, O);
  if (!plain || dbias != nullptr) {
    MOE_LAUNCH((linear_dz_kernel<T>), dim3((O + 255) / 256, slots), dim3(256), 0, stream, T_, O, g.act,
               plain ? nullptr : (const T*)z, (const T*)mul, (const T*)dy, (T*)dz, (T*)dmul,
               dbias != nullptr ? ws : nullptr);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (dx == nullptr && dw == nullptr && dbias == nullptr) return hipSuccess;
  const void* d = plain ? dy : dz;
  const Plan2& p = bwd_cuts(T_, I, O, sizeof(T), dx != nullptr, dw != nullptr);
  LinearProduct gx{{T_, I, d, O, g.w, O, nullptr}, O, kActNone, nullptr, nullptr, dx_add, nullptr, dx, p.x.slice, nullptr};
  LinearProduct gw{{I, O, g.x, I, d, O, nullptr}, T_, kActNone, nullptr, nullptr, nullptr, nullptr, dw, p.w.slice, nullptr};
  const ColumnSum sum{ws, slots, O, dbias};
  char* at = (char*)ws + dbias_bytes(T_, O);
  if (p.x.slices > 1) gx.part = (float*)at;
  at += slice_bytes(T_, I, p.x);
  if (p.w.slices > 1) gw.part = (float*)at;
  auto run = [&](auto tx, auto tw) {
    using CX = decltype(tx);
    using CW = decltype(tw);
    const bool tail = (dx != nullptr && has_tail<T, true, true, CX>(gx)) ||
                      (dw != nullptr && has_tail<T, false, false, CW>(gw));
    return tail ? run_bwd<T, CX, CW, true>(gx, gw, sum, p, stream)
                : run_bwd<T, CX, CW, false>(gx, gw, sum, p, stream);
  };
  hipError_t err = hipErrorUnknown;
  if constexpr (sizeof(T) == 2) {
    if (p.pair == 0) err = run(Tile0{}, Tile0{});
    if (p.pair == 1) err = run(Tile0{}, Tile1{});
    if (p.pair == 2) err = run(Tile1{}, Tile0{});
    if (p.pair == 3) err = run(Tile1{}, Tile1{});
  }
  if (p.pair == 4) err = run(Tile2{}, Tile2{});
  if (p.pair == 5) err = run(Tile3{}, Tile3{});
  if (p.pair == 6) err = run(Tile4<T>{}, Tile4<T>{});
  if (p.pair == 7) err = run(Tile5{}, Tile4<T>{});
  if (err != hipSuccess) return err;
  return add_slices<T>(gx, gw, stream);
}

}  // namespace

// The partials of any call with these sizes: the forward's slices, or the
// backward's column sums and both products' slices (either product may be left out).
size_t linear_workspace_bytes(int T, int I, int O, int esize) {
  return remembered<size_t>(T, I, O, esize + 32, [&] {
    size_t need = slice_bytes(T, O, fwd_cut(T, I, O, esize));
    for (int want = 0; want < 4; ++want) {
      const Plan2& p = bwd_cuts(T, I, O, esize, want & 1, want & 2);
      need = std::max(need, dbias_bytes(T, O) + slice_bytes(T, I, p.x) + slice_bytes(I, O, p.w));
    }
    return need;
  });
}

bool linear_fwd_splits(int T, int I, int O, int esize) { return fwd_cut(T, I, O, esize).slices > 1; }

hipError_t launch_linear_fwd(const LinearArgs& g, int esize, const void* bias, const void* mul, const void* residual,
                             void* z, void* y, void* ws, hipStream_t stream) {
  const LinearProduct p{{g.T, g.O, g.x, g.I, g.w, g.O, nullptr}, g.I, g.act, bias, mul, residual, z, y, 0, nullptr};
  return esize == 4 ? linear_fwd_typed<float>(p, (float*)ws, stream)
                    : linear_fwd_typed<uint16_t>(p, (float*)ws, stream);
}

hipError_t launch_linear_bwd(const LinearArgs& g, int esize, const void* z, const void* mul, const void* dy, void* dz,
                             const void* dx_add, void* dx, void* dw, void* dbias, void* dmul, void* ws,
                             hipStream_t stream) {
  return esize == 4 ? linear_bwd_typed<float>(g, z, mul, dy, dz, dx_add, dx, dw, dbias, dmul, (float*)ws, stream)
                    : linear_bwd_typed<uint16_t>(g, z, mul, dy, dz, dx_add, dx, dw, dbias, dmul, (float*)ws, stream);
}

}  // namespace moe
