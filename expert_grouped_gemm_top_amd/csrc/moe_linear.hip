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
#include "moe_lds32.h"
#include "moe_rows.h"

namespace moe {

namespace {

enum Act { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

constexpr float kTanhA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

// exp(v) and 1 / (1 + exp(-v)) on the hardware's exp2 and reciprocal: relative
// errors of at most (1.5 |v| + 2) 2^-24 and of that share of exp(-v) plus 2^-22
// (the library's expf, erfcf and division took 7 of 28 us of a GELU product's
// epilogue at 4099 x 768).
__device__ __forceinline__ float quick_exp(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504f); }
__device__ __forceinline__ float logistic(float v) { return __builtin_amdgcn_rcpf(1.0f + quick_exp(-v)); }

// Phi(z), the normal distribution: erfc(|z| / sqrt 2) / 2 by formula 7.1.26 of
// Abramowitz and Stegun, erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2), t = 1 / (1 + p x),
// |error| <= 1.5e-7, mirrored for z > 0.
__device__ __forceinline__ float normal_cdf(float z) {
  const float x = fabsf(z) * 0.70710678f;
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * x);
  const float poly =
      t * (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
  const float tail = 0.5f * poly * quick_exp(-x * x);
  return z > 0.0f ? 1.0f - tail : tail;
}

// act(z); NaN stays NaN.
__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;
    case kActGelu: return z * normal_cdf(z);
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
      const float phi = normal_cdf(c);
      value = z * phi;
      slope = phi + c * 0.3989422804014327f * quick_exp(-0.5f * c * c);
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

// C [M, N] = A B over K, then the epilogue.  Either operand may lie with k
// contiguous ("KC": a[m lda + k], b[n ldb + k]) or with its own index contiguous
// (a[k lda + m], b[k ldb + n]).
struct LinearProduct {
  int M, N, K;
  const void* a;
  int64_t lda;
  const void* b;
  int64_t ldb;
  int act;
  const void *bias, *mul, *residual;
  void *z, *out;
  int slice;    // k per slice of a split reduction, a multiple of the kernels' stage depth (>= K: not split)
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
  if (g.act != kActNone) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = act_value(g.act, v[j]);
  }
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
__device__ __forceinline__ void leave8(const LinearProduct& g, int slice, int64_t m, int n, float (&v)[8]) {
  if (g.part != nullptr) store8(g.part + ((int64_t)slice * g.M + m) * g.N + n, v);
  else finish8<T>(g, m, n, v);
}

// Adds the slices of a split reduction in order, then the epilogue.
template <typename T>
__global__ __launch_bounds__(256) void linear_slices_kernel(LinearProduct g, int slices) {
  const int runs = g.N / 8;
  const int64_t total = (int64_t)g.M * runs, MN = (int64_t)g.M * g.N;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
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

// Row and column tile of workgroup `wg`: each XCD walks a contiguous range of
// the tiles; groups of up to `depth` row tiles x all column tiles, column-major
// within a group, so that tiles resident together share operands in L2.
__device__ __forceinline__ void tile_of(int wg, int mtiles, int ntiles, int depth, int& mt, int& nt) {
  const int item = xcd_item(wg, mtiles * ntiles);
  const int grp = item / (depth * ntiles), within = item - grp * depth * ntiles;
  const int gm = min(depth, mtiles - depth * grp);
  mt = depth * grp + within % gm;
  nt = within / gm;
}

// ---- bf16 on the 32x32x16 matrix core ------------------------------------------

// 16-byte chunk position in a [row][64 k] LDS tile (128-byte rows): 16 rows of
// one fragment read fall in distinct bank groups.
__device__ __forceinline__ int kc_key(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// k row of a [k][ROWS] LDS tile -> XOR on the 16-byte chunk index: the 4 k rows x
// 4 chunks that half a wave's transpose read covers lie in distinct banks
// (256-byte rows and longer: every row starts at the same bank; 128-byte rows: every other one).
template <int ROWS>
__device__ __forceinline__ int nc_key(int k) {
  static_assert(ROWS >= 64, "eight chunks at least");
  return ROWS >= 128 ? 4 * (k & 3) : 4 * ((k >> 1) & 1);
}

// 32x32x16 operand fragment of rows row0 .. row0 + 31, k 16 sub .. + 15, from a
// [k][ROWS] tile: in 16-lane group G, lane r points at k 8 (G >> 1) + 4 h +
// (r >> 2) and rows 16 (G & 1) + 4 (r & 3) .. + 3, and receives 4 consecutive k of one
// row (half of its 8).
template <int ROWS>
__device__ __forceinline__ u32x4 nc_frag(const unsigned char* tile, int sub, int row0) {
  const int l = __lane_id(), G = l >> 4, r = l & 15;
  const int row = row0 + 16 * (G & 1) + 4 * (r & 3);
  v4i16 part[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = 16 * sub + 8 * (G >> 1) + 4 * h + (r >> 2);
    part[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_v4i16*)(tile + k * (2 * ROWS) + 16 * ((row >> 3) ^ nc_key<ROWS>(k)) + 2 * (row & 7)));
  }
  const u32x2 lo = __builtin_bit_cast(u32x2, part[0]), hi = __builtin_bit_cast(u32x2, part[1]);
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// One operand's stage: ROWS x BK elements by direct global->LDS loads, INS per
// wave.  KC: LDS [row][BK]; otherwise LDS [BK][ROWS].  Chunks outside the
// operand come from zeros (TAIL; rows of a KC operand past its end re-read the
// last row and reach only outputs that are not stored).
template <bool KC, int ROWS, int BK, int NW, bool TAIL>
struct Loader {
  static constexpr int INS = ROWS * BK * 2 / 1024 / NW;
  static_assert(ROWS * BK * 2 == INS * 1024 * NW, "whole loads");
  const uint16_t* src[INS];
  int k[INS];    // k of this lane's chunk within the stage
  bool ok[INS];  // inside the operand's rows
  int64_t step;  // elements per k
  __device__ void init(const void* base, int64_t ld, int r0, int rows, int w, int l) {
    step = KC ? 1 : ld;
#pragma unroll
    for (int i = 0; i < INS; ++i) {
      if (KC) {
        const int row = (512 / BK) * (INS * w + i) + l / (BK / 8);
        const int chunk = kc_key(row, l % (BK / 8));
        k[i] = 8 * chunk;
        ok[i] = true;
        src[i] = (const uint16_t*)base + (int64_t)min(r0 + row, rows - 1) * ld + 8 * chunk;
      } else {
        k[i] = (512 / ROWS) * (INS * w + i) + l / (ROWS / 8);
        const int c = r0 + 8 * ((l % (ROWS / 8)) ^ nc_key<ROWS>(k[i]));
        ok[i] = c < rows;
        src[i] = (const uint16_t*)base + (int64_t)k[i] * ld + (ok[i] ? c : 0);
      }
    }
  }
  __device__ void issue(int k0, int K, unsigned char* tile, int w) const {
#pragma unroll
    for (int i = 0; i < INS; ++i) {
      const uint16_t* p = src[i] + k0 * step;
      if (TAIL && (!ok[i] || k0 + k[i] >= K)) p = zero_chunk();
      g2lds(p, tile + 1024 * (INS * w + i));
    }
  }
};

template <bool KC, int ROWS, int BK>
__device__ __forceinline__ u32x4 tile_frag(const unsigned char* tile, int sub, int row0) {
  if (KC) {
    const int row = row0 + (__lane_id() & 31);
    return *(const u32x4*)(tile + row * (2 * BK) + 16 * kc_key(row, 2 * sub + (__lane_id() >> 5)));
  } else {
    return nc_frag<ROWS>(tile, sub, row0);
  }
}

// Workgroup = BM x BN outputs by KG groups of NW waves, each group laid out
// WM x (NW / WM) over the tile and taking every KG-th 64 k of the reduction
// (the groups' sums are added at the end): two waves on a SIMD hide each other's
// LDS reads and waits without a smaller wave tile.  STAGES LDS stages of KG x
// 64 k.  A stage is waited for before the last 16 k of the one in front, so
// its first fragments are read under those products, and its successor's loads
// go out in two halves before the next two runs of products.
template <bool AKC, bool BKC, int BM, int BN, int NW, int WM, int KG, int STAGES, bool TAIL>
__global__ __launch_bounds__(64 * NW * KG, NW * KG / 4) void linear_tile_kernel(LinearProduct g, int depth) {
  constexpr int BK = 64, SUBS = BK / 16;
  constexpr int TM = BM / WM, TN = BN / (NW / WM), MI = TM / 32, NJ = TN / 32;
  constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, GROUP = A_BYTES + B_BYTES, STAGE = KG * GROUP;
  extern __shared__ __attribute__((aligned(16))) unsigned char s_dyn[];
  const int tid = threadIdx.x, l = tid & 63, l32 = l & 31, hk = l >> 5;
  const int kg = (tid >> 6) / NW, w = (tid >> 6) % NW;
  const int wm = w % WM, wn = w / WM;
  int mt, nt;
  tile_of(blockIdx.x, (g.M + BM - 1) / BM, (g.N + BN - 1) / BN, depth, mt, nt);
  const int m0 = mt * BM, n0 = nt * BN;
  const int kb = blockIdx.y * g.slice, ke = min(g.K, kb + g.slice);

  Loader<AKC, BM, BK, NW, TAIL> la;
  Loader<BKC, BN, BK, NW, TAIL> lb;
  la.init(g.a, g.lda, m0, g.M, w, l);
  lb.init(g.b, g.ldb, n0, g.N, w, l);
  constexpr int INS = Loader<AKC, BM, BK, NW, TAIL>::INS + Loader<BKC, BN, BK, NW, TAIL>::INS;  // loads of a stage
  // stage s lies in buffer s % STAGES; a group loads and reads its own part of it
  unsigned char* const mine = s_dyn + kg * GROUP;
  auto issue_a = [&](int s, int buf) { la.issue(kb + (s * KG + kg) * BK, ke, mine + buf * STAGE, w); };
  auto issue_b = [&](int s, int buf) { lb.issue(kb + (s * KG + kg) * BK, ke, mine + buf * STAGE + A_BYTES, w); };

  f32x16 acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  struct Frags {
    u32x4 a[MI], b[NJ];
  };
  auto products = [&](const Frags& cur, const unsigned char* st, int next_sub, Frags& nxt) {
    __builtin_amdgcn_s_setprio(1);
    if (next_sub >= 0) {
#pragma unroll
      for (int i = 0; i < MI; ++i) nxt.a[i] = tile_frag<AKC, BM, BK>(st, next_sub, TM * wm + 32 * i);
#pragma unroll
      for (int j = 0; j < NJ; ++j) nxt.b[j] = tile_frag<BKC, BN, BK>(st + A_BYTES, next_sub, TN * wn + 32 * j);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < MI; ++i) acc[i][j] = mfma32(cur.b[j], cur.a[i], acc[i][j]);
    constexpr int READS = ((AKC ? 1 : 2) * MI + (BKC ? 1 : 2) * NJ + MI * NJ - 1) / (MI * NJ);
#pragma unroll
    for (int q = 0; q < MI * NJ; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);      // one product
      __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);  // its share of the LDS reads
    }
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };

  const int steps = (ke - kb + KG * BK - 1) / (KG * BK);
  static_assert(SUBS == 4, "four runs of products per stage");
  Frags f0, f1;
  for (int s = 0; s < STAGES - 1 && s < steps; ++s) {
    issue_a(s, s);
    issue_b(s, s);
  }
  if (steps >= STAGES - 1) wait_vmcnt<(STAGES - 2) * INS>();  // stage 0 has landed, later ones need not have
  else wait_vmcnt<0>();
  barrier_no_fence();
  if (steps > STAGES - 1) {
    issue_a(STAGES - 1, STAGES - 1);
    issue_b(STAGES - 1, STAGES - 1);
  }
#pragma unroll
  for (int i = 0; i < MI; ++i) f0.a[i] = tile_frag<AKC, BM, BK>(mine, 0, TM * wm + 32 * i);
#pragma unroll
  for (int j = 0; j < NJ; ++j) f0.b[j] = tile_frag<BKC, BN, BK>(mine + A_BYTES, 0, TN * wn + 32 * j);
  products(f0, mine, 1, f1);
  products(f1, mine, 2, f0);
  products(f0, mine, 3, f1);
  int buf = 0;  // of stage s - 1, which stage s + STAGES - 1 takes over
  for (int s = 1; s < steps; ++s) {
    const int next = buf + 1 < STAGES ? buf + 1 : 0;
    const unsigned char* st = mine + next * STAGE;
    // stage s has landed; of the stages behind it, STAGES - 2 may be in flight
    if (STAGES > 2 && s + STAGES - 2 < steps) wait_vmcnt<(STAGES - 2) * INS>();
    else wait_vmcnt<0>();
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's reads of stage s - 1 are done
    barrier_no_fence();                   // ... and every wave's: its buffer can be loaded again
    const bool more = s + STAGES - 1 < steps;
    if (more) issue_a(s + STAGES - 1, buf);
    products(f1, st, 0, f0);
    if (more) issue_b(s + STAGES - 1, buf);
    products(f0, st, 1, f1);
    products(f1, st, 2, f0);
    products(f0, st, 3, f1);
    buf = next;
  }
  products(f1, mine, -1, f0);

  // The fp32 tile leaves through the idle stage buffers, HC columns at a time
  // ([row][HC], 16-byte chunk c of row r at c ^ (r & 15)), so that the epilogue
  // reads and writes runs of eight neighbouring outputs.  Register r of
  // acc[i][j] is row TM wm + 32 i + l32, column TN wn + 32 j + 8 (r / 4) + 4 hk + r % 4.
  constexpr int FIT = STAGES * STAGE / (BM * 4);
  constexpr int HC = FIT >= BN ? BN : (FIT >= 128 ? 128 : 64);
  static_assert(BM * HC * 4 <= STAGES * STAGE && HC % TN == 0 && BN % HC == 0, "staging");
  float* s_f = reinterpret_cast<float*>(s_dyn);
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's last fragment reads are done
#pragma unroll
  for (int part = 0; part < BN / HC; ++part) {
    barrier_no_fence();  // every wave is done with the stage buffers / the previous part
#pragma unroll
    for (int k2 = 0; k2 < KG; ++k2) {  // the groups in turn: the first writes its sums, the others add theirs
      if (kg == k2 && TN * wn / HC == part) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int row = TM * wm + 32 * i + l32, col = TN * wn - HC * part + 32 * j + 8 * q + 4 * hk;
              f32x4* at = (f32x4*)(s_f + row * HC + 4 * ((col >> 2) ^ (row & 15)));
              f32x4 v = f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
              if (k2 > 0) v += *at;
              *at = v;
            }
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the staged values are written
      barrier_no_fence();
    }
#pragma unroll 2
    for (int it = tid; it < BM * HC / 8; it += 64 * NW * KG) {
      const int row = it / (HC / 8), c8 = it % (HC / 8);
      const int m = m0 + row, n = n0 + HC * part + 8 * c8;
      if (m >= g.M || n >= g.N) continue;  // N is a multiple of 8: a run is all in or all out
      const f32x4 lo = *(const f32x4*)(s_f + row * HC + 4 * ((2 * c8) ^ (row & 15)));
      const f32x4 hi = *(const f32x4*)(s_f + row * HC + 4 * ((2 * c8 + 1) ^ (row & 15)));
      float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      leave8<uint16_t>(g, blockIdx.y, m, n, v);
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's reads of the staged rows are done
  }
}

// ---- fp32 on the 32x32x2 matrix core ---------------------------------------------

// D = first x second + D: lane l supplies row / column l % 32 of k = l / 32; the
// registers of D lie as for mfma32.
__device__ __forceinline__ f32x16 mfma32_f32(float first, float second, f32x16 acc) {
  return __builtin_amdgcn_mfma_f32_32x32x2f32(first, second, acc, 0, 0, 0);
}

// Workgroup = BT x BT outputs, four waves of (BT / 2)^2, 16 k per LDS stage, the
// next stage's values loaded into registers under the products.
template <bool AKC, bool BKC, int BT>
__global__ __launch_bounds__(256) void linear_f32_kernel(LinearProduct g, int depth) {
  constexpr int BK = 16, PITCH = BT + 32, NB = BT / 64;  // 32 x 32 blocks per wave side
  constexpr int QUADS = BT * BK / 4 / 256;               // 16-byte loads per thread and operand
  __shared__ __attribute__((aligned(16))) float s_a[BK * PITCH], s_b[BK * PITCH];
  const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, l32 = l & 31, hk = l >> 5;
  const int wm = w & 1, wn = w >> 1;
  int mt, nt;
  tile_of(blockIdx.x, (g.M + BT - 1) / BT, (g.N + BT - 1) / BT, depth, mt, nt);
  const int m0 = mt * BT, n0 = nt * BT;
  const int kb = blockIdx.y * g.slice, ke = min(g.K, kb + g.slice);
  f32x4 ra[QUADS], rb[QUADS];
  // four neighbouring elements of an operand; those outside are zero (the contiguous extent is a multiple of 4)
  auto fetch = [&](auto kc, const void* base, int64_t ld, int r0, int rows, int k0, f32x4 (&v)[QUADS]) {
#pragma unroll
    for (int i = 0; i < QUADS; ++i) {
      const int q = tid + 256 * i;
      int r, k;
      if constexpr (decltype(kc)::value) {
        r = r0 + q / (BK / 4);
        k = k0 + 4 * (q % (BK / 4));
      } else {
        k = k0 + q / (BT / 4);
        r = r0 + 4 * (q % (BT / 4));
      }
      const bool in = r < rows && k < ke;
      const int64_t at = decltype(kc)::value ? r * ld + k : k * ld + r;
      v[i] = in ? *(const f32x4*)((const float*)base + at) : f32x4{0.f, 0.f, 0.f, 0.f};
    }
  };
  auto put = [&](auto kc, float* s, const f32x4 (&v)[QUADS]) {
#pragma unroll
    for (int i = 0; i < QUADS; ++i) {
      const int q = tid + 256 * i;
      if constexpr (decltype(kc)::value) {
        const int r = q / (BK / 4), k = 4 * (q % (BK / 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) s[(k + j) * PITCH + r] = v[i][j];
      } else {
        *(f32x4*)(s + (q / (BT / 4)) * PITCH + 4 * (q % (BT / 4))) = v[i];
      }
    }
  };
  using A = std::integral_constant<bool, AKC>;
  using B = std::integral_constant<bool, BKC>;
  f32x16 acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  fetch(A{}, g.a, g.lda, m0, g.M, kb, ra);
  fetch(B{}, g.b, g.ldb, n0, g.N, kb, rb);
  for (int k0 = kb; k0 < ke; k0 += BK) {
    put(A{}, s_a, ra);
    put(B{}, s_b, rb);
    __syncthreads();
    if (k0 + BK < ke) {
      fetch(A{}, g.a, g.lda, m0, g.M, k0 + BK, ra);
      fetch(B{}, g.b, g.ldb, n0, g.N, k0 + BK, rb);
    }
#pragma unroll
    for (int k = 0; k < BK; k += 2) {
      float fa[NB], fb[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        fa[i] = s_a[(k + hk) * PITCH + 32 * (NB * wm + i) + l32];
        fb[i] = s_b[(k + hk) * PITCH + 32 * (NB * wn + i) + l32];
      }
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < NB; ++i) acc[i][j] = mfma32_f32(fb[j], fa[i], acc[i][j]);
    }
    __syncthreads();
  }
  // lane pairs l, l + 32 hold the two halves of eight neighbouring columns of one
  // row: they swap quads so that each holds whole runs
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int m = m0 + 32 * (NB * wm + i) + l32;
        const int n = n0 + 32 * (NB * wn + j) + 16 * p + 8 * hk;
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // quads 2 p (columns + 0..7) and 2 p + 1 (columns + 8..15): lane half 0 keeps the first run, half 1 the second
          const float mine0 = acc[i][j][8 * p + e], mine1 = acc[i][j][8 * p + 4 + e];
          const float give = hk ? mine0 : mine1;
          const float got = __shfl_xor(give, 32, kWave);
          v[e] = hk ? got : mine0;
          v[4 + e] = hk ? mine1 : got;
        }
        if (m < g.M && n < g.N) leave8<float>(g, blockIdx.y, m, n, v);
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

// ---- launchers -------------------------------------------------------------------

template <typename T>
hipError_t add_slices(const LinearProduct& g, hipStream_t stream) {
  const int slices = (g.K + g.slice - 1) / g.slice;
  const int64_t runs = (int64_t)g.M * (g.N / 8);
  MOE_LAUNCH((linear_slices_kernel<T>), dim3((unsigned)std::min<int64_t>((runs + 255) / 256, 4096)), dim3(256), 0,
             stream, g, slices);
  return hipGetLastError();
}

// The workgroup tiles, largest first, and what a pass of them over the chip's
// 256 CUs takes: `step` us per 64 k (`step_few` when at most 160 workgroups run), `round` us for its prologue
// and epilogue.  Measured on one MI355X with grids of 128, 256 and 512
// workgroups and reductions of 512, 2048 and 4096 (all three operand layouts
// within 8 %).  A larger tile moves fewer bytes through LDS per product (at 256
// workgroups: 256 x 256 1.32 PFLOP/s, 256 x 128 1.14, 128 x 128 1.01, 128 x 64 0.84, 64 x 64 0.61) but
// leaves CUs idle where the outputs are few: 4099 x 768 over 2048 takes 49 us
// on 256 x 256, 30 on 256 x 128, 20.9 on 128 x 128, 25.8 on 128 x 64 tiles.
struct TileCost {
  int bm, bn;
  double step, step_few, round;
};
enum { kTile256x256 = 0, kTile256x128, kTile128x128, kTile128x64, kTile64x64, kTilesBf16 };
constexpr TileCost kCostBf16[kTilesBf16] = {
    {256, 256, 1.62, 1.13, 8.5}, {256, 128, 0.94, 0.74, 4.5}, {128, 128, 0.53, 0.47, 2.6},
    {128, 64, 0.33, 0.27, 2.0},  {64, 64, 0.22, 0.19, 1.0}};
// fp32: the same per 16 k
enum { kTileF128 = 0, kTileF64, kTilesF32 };
constexpr TileCost kCostF32[kTilesF32] = {{128, 128, 1.10, 1.10, 4.0}, {64, 64, 0.35, 0.30, 2.0}};

constexpr double kLaunchUs = 3.5;              // one more kernel behind another
constexpr double kSliceBytesPerUs = 4.0e6;     // partials written and read again

// What runs a product: the tile, and the slices of its reduction.
struct Plan {
  int tile;
  int slices;
  int slice;  // k per slice
};

// The plan of least estimated time.  Splitting the reduction pays where few
// tiles meet a long reduction: 2048 x 768 outputs over 4099 rows take 56 us on
// 128 x 128 tiles, 31 us in two slices with the sum behind them.
Plan plan_of(int M, int N, int K, int esize) {
  constexpr int kCus = 256, kFew = 160;
  const bool bf16 = esize == 2;
  const int stage = bf16 ? 64 : 16, grain = bf16 ? 128 : 16;
  Plan best{};
  double best_us = 0.0;
  for (int c = 0; c < (bf16 ? (int)kTilesBf16 : (int)kTilesF32); ++c) {
    const TileCost& t = bf16 ? kCostBf16[c] : kCostF32[c];
    const int64_t tiles = (int64_t)((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
    for (int want : {1, 2, 3, 4, 6, 8, 12, 16}) {
      const int slice = ((K + want - 1) / want + grain - 1) / grain * grain;
      const int slices = (K + slice - 1) / slice;
      if (want > 1 && (slices == 1 || tiles * want > 2 * kCus)) break;
      const int64_t groups = tiles * slices, rest = groups % kCus;
      const double steps = (double)((std::min(K, slice) + stage - 1) / stage);
      double us = kLaunchUs + (double)(groups / kCus) * (steps * t.step + t.round);
      if (rest > 0) us += steps * (rest > kFew ? t.step : t.step_few) + t.round;
      if (slices > 1) us += kLaunchUs + (double)slices * M * N * 8.0 / kSliceBytesPerUs;
      if (best.slices == 0 || us < best_us) {
        best = Plan{c, slices, slice};
        best_us = us;
      }
    }
  }
  return best;
}

size_t plan_bytes(int M, int N, int K, int esize) {
  const Plan p = plan_of(M, N, K, esize);
  return p.slices > 1 ? (size_t)p.slices * M * N * sizeof(float) : 0;
}

template <bool AKC, bool BKC, int BM, int BN, int NW, int WM, int KG, int STAGES, bool TAIL>
hipError_t launch_tiles(const LinearProduct& g, int slices, hipStream_t stream) {
  constexpr size_t lds = (size_t)STAGES * KG * (BM + BN) * 64 * 2;
  auto kern = linear_tile_kernel<AKC, BKC, BM, BN, NW, WM, KG, STAGES, TAIL>;
  static PerDeviceOnce once;
  hipError_t err = allow_dynamic_lds(once, (const void*)kern, lds);
  if (err != hipSuccess) return err;
  const int64_t tiles = (int64_t)((g.M + BM - 1) / BM) * ((g.N + BN - 1) / BN);
  MOE_LAUNCH(kern, dim3((unsigned)tiles, slices), dim3(64 * NW * KG), lds, stream, g, 1024 / BM);
  return hipGetLastError();
}

template <bool AKC, bool BKC, int BM, int BN, int NW, int WM, int KG, int STAGES>
hipError_t launch_bf16(const LinearProduct& g, int slices, hipStream_t stream) {
  // whole stages, in every slice: nothing to mask (a stage that ran past the reduction's end would read past the operands)
  const bool tail = g.K % (64 * KG) != 0 || (slices > 1 && g.slice % (64 * KG) != 0) || (!BKC && g.N % BN != 0) || (!AKC && g.M % BM != 0);
  return tail ? launch_tiles<AKC, BKC, BM, BN, NW, WM, KG, STAGES, true>(g, slices, stream)
              : launch_tiles<AKC, BKC, BM, BN, NW, WM, KG, STAGES, false>(g, slices, stream);
}

// AKC, BKC: which operands have k contiguous.
template <typename T, bool AKC, bool BKC>
hipError_t product(LinearProduct g, float* ws, hipStream_t stream) {
  const Plan p = plan_of(g.M, g.N, g.K, sizeof(T));
  g.slice = p.slice;
  g.part = p.slices > 1 ? ws : nullptr;
  hipError_t err;
  if constexpr (std::is_same<T, float>::value) {
    const int bt = kCostF32[p.tile].bm;
    const dim3 grid((unsigned)((int64_t)((g.M + bt - 1) / bt) * ((g.N + bt - 1) / bt)), p.slices);
    if (p.tile == kTileF128) MOE_LAUNCH((linear_f32_kernel<AKC, BKC, 128>), grid, dim3(256), 0, stream, g, 8);
    else MOE_LAUNCH((linear_f32_kernel<AKC, BKC, 64>), grid, dim3(256), 0, stream, g, 8);
    err = hipGetLastError();
  } else {
    switch (p.tile) {
      case kTile256x256: err = launch_bf16<AKC, BKC, 256, 256, 8, 2, 1, 2>(g, p.slices, stream); break;
      case kTile256x128: err = launch_bf16<AKC, BKC, 256, 128, 8, 4, 1, 3>(g, p.slices, stream); break;
      case kTile128x128: err = launch_bf16<AKC, BKC, 128, 128, 4, 2, 2, 2>(g, p.slices, stream); break;
      case kTile128x64: err = launch_bf16<AKC, BKC, 128, 64, 4, 2, 2, 3>(g, p.slices, stream); break;
      default: err = launch_bf16<AKC, BKC, 64, 64, 4, 2, 2, 4>(g, p.slices, stream); break;
    }
  }
  if (err != hipSuccess || p.slices == 1) return err;
  return add_slices<T>(g, stream);
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
    LinearProduct p{T_, I, O, d, O, g.w, O, kActNone, nullptr, nullptr, dx_add, nullptr, dx, 0, nullptr};
    hipError_t err = product<T, true, true>(p, ws, stream);
    if (err != hipSuccess) return err;
  }
  if (dw != nullptr) {
    LinearProduct p{I, O, T_, g.x, I, d, O, kActNone, nullptr, nullptr, nullptr, nullptr, dw, 0, nullptr};
    return product<T, false, false>(p, ws, stream);
  }
  return hipSuccess;
}

}  // namespace

// The partials of one launch at a time: a backward's column sums, then each product's slices.
size_t linear_workspace_bytes(int T, int I, int O, int esize) {
  return std::max({(size_t)dz_slots(T, O) * O * sizeof(float), plan_bytes(T, O, I, esize), plan_bytes(T, I, O, esize),
                   plan_bytes(I, O, T, esize)});
}

hipError_t launch_linear_fwd(const LinearArgs& g, int esize, const void* bias, const void* mul, const void* residual,
                             void* z, void* y, void* ws, hipStream_t stream) {
  const LinearProduct p{g.T, g.O, g.I, g.x, g.I, g.w, g.O, g.act, bias, mul, residual, z, y, 0, nullptr};
  return esize == 4 ? product<float, true, false>(p, (float*)ws, stream)
                    : product<uint16_t, true, false>(p, (float*)ws, stream);
}

hipError_t launch_linear_bwd(const LinearArgs& g, int esize, const void* z, const void* mul, const void* dy, void* dz,
                             const void* dx_add, void* dx, void* dw, void* dbias, void* dmul, void* ws,
                             hipStream_t stream) {
  return esize == 4 ? linear_bwd_typed<float>(g, z, mul, dy, dz, dx_add, dx, dw, dbias, dmul, (float*)ws, stream)
                    : linear_bwd_typed<uint16_t>(g, z, mul, dy, dz, dx_add, dx, dw, dbias, dmul, (float*)ws, stream);
}

}  // namespace moe
