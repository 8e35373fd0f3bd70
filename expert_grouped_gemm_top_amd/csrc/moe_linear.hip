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
#include "moe_lds32.h"
#include "moe_linear_plan.h"
#include "moe_rows.h"

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
__device__ __forceinline__ void leave8(const LinearProduct& g, int slice, int64_t m, int n, float (&v)[8]) {
  if (g.part != nullptr) store8(g.part + ((int64_t)slice * g.M + m) * g.N + n, v);
  else finish8<T>(g, m, n, v);
}

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

// ---- one workgroup tile on the matrix cores ---------------------------------------

// Both types lie alike in LDS: a stage is 128 bytes of k (64 bf16, 32 fp32), a
// fragment 16 bytes per lane (8 bf16 or 4 fp32 k of one row), and a run of
// products takes two fragments' k: one 32x32x16 bf16 product, or four 32x32x2
// fp32 ones, the j-th over element j of both lanes' fragments.
template <typename T>
constexpr int kChunk = 16 / (int)sizeof(T);
template <typename T>
constexpr int kStageK = 128 / (int)sizeof(T);
template <typename T>
constexpr int kRunProducts = sizeof(T) == 2 ? 1 : 4;

// The q-th product of a run.
template <typename T>
__device__ __forceinline__ f32x16 product32(u32x4 first, u32x4 second, int q, f32x16 acc) {
  if constexpr (sizeof(T) == 2) return mfma32(first, second, acc);
  else
    return __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(first[q]), __uint_as_float(second[q]), acc, 0, 0, 0);
}

// 16-byte chunk position in a [row][stage k] LDS tile (128-byte rows): 16 rows of
// one fragment read fall in distinct bank groups.
__device__ __forceinline__ int kc_key(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// k row of a [k][ROWS] LDS tile -> XOR on the 16-byte chunk index.  bf16: the 4 k
// rows x 4 chunks that half a wave's transpose read covers lie in distinct banks
// (256-byte rows and longer: every row starts at the same bank; 128-byte rows: every
// other one; 64-byte rows need no key).  fp32: the two k rows, 4 apart, of a wave's
// read (128-byte rows, where a key cannot part them: their places, nc_place).
template <typename T, int ROWS>
__device__ __forceinline__ int nc_key(int k) {
  if (ROWS == 32) return 0;
  if (sizeof(T) == 4) return 8 * ((k >> 2) & 1);
  return ROWS >= 128 ? 4 * (k & 3) : 4 * ((k >> 1) & 1);
}
template <typename T, int ROWS>
__device__ __forceinline__ int nc_place(int k) { return ROWS == 32 && sizeof(T) == 4 ? k ^ ((k >> 2) & 1) : k; }

// Fragment of rows row0 .. row0 + 31, run `sub` of the stage's four, from a
// [k][ROWS] tile.  bf16, k 16 sub .. + 15: in 16-lane group G, lane r points at k
// 8 (G >> 1) + 4 h + (r >> 2) and rows 16 (G & 1) + 4 (r & 3) .. + 3, and receives 4
// consecutive k of one row (half of its 8).  fp32, k 8 sub .. + 7: lane l reads k
// 4 (l / 32) + j of row l % 32.
template <typename T, int ROWS>
__device__ __forceinline__ u32x4 nc_frag(const unsigned char* tile, int sub, int row0) {
  const int l = __lane_id(), G = l >> 4, r = l & 15;
  if constexpr (sizeof(T) == 4) {
    const int row = row0 + (l & 31), k = 8 * sub + 4 * (l >> 5);
    const unsigned char* col = tile + 16 * ((row >> 2) ^ nc_key<T, ROWS>(k)) + 4 * (row & 3);
    const unsigned char* even = col + nc_place<T, ROWS>(k) * (4 * ROWS);
    const unsigned char* odd = col + nc_place<T, ROWS>(k + 1) * (4 * ROWS);
    return u32x4{*(const uint32_t*)even, *(const uint32_t*)odd, *(const uint32_t*)(even + 8 * ROWS),
                 *(const uint32_t*)(odd + 8 * ROWS)};
  }
  const int row = row0 + 16 * (G & 1) + 4 * (r & 3);
  v4i16 part[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = 16 * sub + 8 * (G >> 1) + 4 * h + (r >> 2);
    part[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_v4i16*)(tile + k * (2 * ROWS) + 16 * ((row >> 3) ^ nc_key<T, ROWS>(k)) + 2 * (row & 7)));
  }
  const u32x2 lo = __builtin_bit_cast(u32x2, part[0]), hi = __builtin_bit_cast(u32x2, part[1]);
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// One operand's stage: ROWS x 128 bytes by direct global->LDS loads, INS per
// wave.  KC: LDS [row][k]; otherwise LDS [k][ROWS].  Chunks outside the
// operand come from zeros (TAIL; rows of a KC operand past its end re-read the
// last row and reach only outputs that are not stored).
template <typename T, bool KC, int ROWS, int NW, bool TAIL>
struct Loader {
  static constexpr int INS = ROWS * 128 / 1024 / NW, CH = kChunk<T>, CHUNKS = ROWS / CH;
  static_assert(ROWS * 128 == INS * 1024 * NW, "whole loads");
  const T* src[INS];
  uint32_t k[INS];  // TAIL: k of this lane's chunk, past any K for rows outside the operand
  int64_t step;     // elements from one stage to the next
  __device__ void init(const void* base, int64_t ld, int r0, int rows, int k0, int stage_k, int w, int l) {
    step = KC ? stage_k : stage_k * ld;
#pragma unroll
    for (int i = 0; i < INS; ++i) {
      if (KC) {
        const int row = 8 * (INS * w + i) + l / 8;
        k[i] = k0 + CH * kc_key(row, l % 8);
        src[i] = (const T*)base + (int64_t)min(r0 + row, rows - 1) * ld + k[i];
      } else {
        const int at = 64 * (INS * w + i) + l;  // chunk of the stage
        const int ks = nc_place<T, ROWS>(at / CHUNKS);  // its own inverse
        const int c = r0 + CH * ((at % CHUNKS) ^ nc_key<T, ROWS>(ks));
        k[i] = k0 + ks;
        src[i] = (const T*)base + (int64_t)k[i] * ld + (c < rows ? c : 0);
        if (c >= rows) k[i] = 0x80000000u;
      }
    }
  }
  // The stages in turn.
  __device__ void issue(int K, int stage_k, unsigned char* tile, int w) {
#pragma unroll
    for (int i = 0; i < INS; ++i) {
      const T* p = src[i];
      if (TAIL && k[i] >= (uint32_t)K) p = reinterpret_cast<const T*>(zero_chunk());
      g2lds(p, tile + 1024 * (INS * w + i));
      src[i] += step;
      if (TAIL) k[i] += stage_k;
    }
  }
};

template <typename T, bool KC, int ROWS>
__device__ __forceinline__ u32x4 tile_frag(const unsigned char* tile, int sub, int row0) {
  if (KC) {
    const int row = row0 + (__lane_id() & 31);
    return *(const u32x4*)(tile + row * 128 + 16 * kc_key(row, 2 * sub + (__lane_id() >> 5)));
  } else {
    return nc_frag<T, ROWS>(tile, sub, row0);
  }
}

// A workgroup tile: BM x BN outputs by KG groups of NW waves, each group laid out
// WM x (NW / WM) over the tile and taking every KG-th 128 bytes of the reduction
// (the groups' sums are added at the end): two waves on a SIMD hide each other's
// LDS reads and waits without a smaller wave tile.  STAGES LDS stages of KG x
// 128 bytes of k.  All have eight waves and mostly a CU's LDS to themselves.
template <int BM_, int BN_, int NW_, int WM_, int KG_, int STAGES_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, NW = NW_, WM = WM_, KG = KG_, STAGES = STAGES_;
  static constexpr int LDS = STAGES * KG * (BM + BN) * 128;
  static_assert(NW * KG == 8 && LDS <= 160 * 1024, "eight waves, one CU's LDS");
};
constexpr int kThreads = 512;

// Output tile `tile` of the product over slice `slice` of its reduction.  A stage
// is waited for before the last run of the one in front, so its first
// fragments are read under those products, and its successor's loads go out in
// two halves before the next two runs of products.
template <typename T, bool AKC, bool BKC, typename C, bool TAIL>
__device__ __forceinline__ void tile_product(const LinearProduct& g, int tile, int slice, unsigned char* s_dyn) {
  constexpr int BM = C::BM, BN = C::BN, NW = C::NW, WM = C::WM, KG = C::KG, STAGES = C::STAGES;
  constexpr int BK = kStageK<T>, RUN = kRunProducts<T>;
  constexpr int TM = BM / WM, TN = BN / (NW / WM), MI = TM / 32, NJ = TN / 32;
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, GROUP = A_BYTES + B_BYTES, STAGE = KG * GROUP;
  const int tid = threadIdx.x, l = tid & 63, l32 = l & 31, hk = l >> 5;
  const int kg = (tid >> 6) / NW, w = (tid >> 6) % NW;
  const int wm = w % WM, wn = w / WM;
  int mt, nt;
  tile_of(tile, (g.M + BM - 1) / BM, (g.N + BN - 1) / BN, 1024 / BM, mt, nt);
  const int m0 = mt * BM, n0 = nt * BN;
  const int kb = slice * g.slice, ke = min(g.K, kb + g.slice);

  Loader<T, AKC, BM, NW, TAIL> la;
  Loader<T, BKC, BN, NW, TAIL> lb;
  la.init(g.a, g.lda, m0, g.M, kb + kg * BK, KG * BK, w, l);
  lb.init(g.b, g.ldb, n0, g.N, kb + kg * BK, KG * BK, w, l);
  constexpr int INS = Loader<T, AKC, BM, NW, TAIL>::INS + Loader<T, BKC, BN, NW, TAIL>::INS;  // loads of a stage
  // stage s lies in buffer s % STAGES; a group loads and reads its own part of it
  unsigned char* const mine = s_dyn + kg * GROUP;
  auto issue_a = [&](int buf) { la.issue(ke, KG * BK, mine + buf * STAGE, w); };
  auto issue_b = [&](int buf) { lb.issue(ke, KG * BK, mine + buf * STAGE + A_BYTES, w); };

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
      for (int i = 0; i < MI; ++i) nxt.a[i] = tile_frag<T, AKC, BM>(st, next_sub, TM * wm + 32 * i);
#pragma unroll
      for (int j = 0; j < NJ; ++j) nxt.b[j] = tile_frag<T, BKC, BN>(st + A_BYTES, next_sub, TN * wn + 32 * j);
    }
#pragma unroll
    for (int q = 0; q < RUN; ++q)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i][j] = product32<T>(cur.b[j], cur.a[i], q, acc[i][j]);
    constexpr int ALL = MI * NJ * RUN, NCR = sizeof(T) == 2 ? 2 : 4;  // products; reads of an NC fragment
    constexpr int READS = ((AKC ? 1 : NCR) * MI + (BKC ? 1 : NCR) * NJ + ALL - 1) / ALL;
#pragma unroll
    for (int q = 0; q < ALL; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);      // one product
      __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);  // its share of the LDS reads
    }
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };

  const int steps = (ke - kb + KG * BK - 1) / (KG * BK);
  Frags f0, f1;
  for (int s = 0; s < STAGES - 1 && s < steps; ++s) {
    issue_a(s);
    issue_b(s);
  }
  if (steps >= STAGES - 1) wait_vmcnt<(STAGES - 2) * INS>();  // stage 0 has landed, later ones need not have
  else wait_vmcnt<0>();
  barrier_no_fence();
  if (steps > STAGES - 1) {
    issue_a(STAGES - 1);
    issue_b(STAGES - 1);
  }
#pragma unroll
  for (int i = 0; i < MI; ++i) f0.a[i] = tile_frag<T, AKC, BM>(mine, 0, TM * wm + 32 * i);
#pragma unroll
  for (int j = 0; j < NJ; ++j) f0.b[j] = tile_frag<T, BKC, BN>(mine + A_BYTES, 0, TN * wn + 32 * j);
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
    if (more) issue_a(buf);
    products(f1, st, 0, f0);
    if (more) issue_b(buf);
    products(f0, st, 1, f1);
    products(f1, st, 2, f0);
    products(f0, st, 3, f1);
    buf = next;
  }
  products(f1, mine, -1, f0);

  // The fp32 tile leaves through the idle stage buffers, HC columns at a time
  // ([row][HC], 16-byte chunk c of row r at c ^ (r mod CH)), so that the epilogue
  // reads and writes runs of eight neighbouring outputs.  Register r of
  // acc[i][j] is row TM wm + 32 i + l32, column TN wn + 32 j + 8 (r / 4) + 4 hk + r % 4.
  constexpr int FIT = STAGES * STAGE / (BM * 4);
  constexpr int HC = FIT >= BN ? BN : (FIT >= 128 ? 128 : 64);
  constexpr int CH = HC / 4 < 16 ? HC / 4 : 16;  // chunks that trade places
  static_assert(BM * HC * 4 <= STAGES * STAGE && HC % TN == 0 && BN % HC == 0, "staging");
  static_assert(KG == 1 || FIT >= KG * BN, "every group's sums in a place of their own");
  float* s_f = reinterpret_cast<float*>(s_dyn);
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's last fragment reads are done
#pragma unroll
  for (int part = 0; part < BN / HC; ++part) {
    barrier_no_fence();  // every wave is done with the stage buffers / the previous part
    if (TN * wn / HC == part) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int row = TM * wm + 32 * i + l32, col = TN * wn - HC * part + 32 * j + 8 * q + 4 * hk;
            *(f32x4*)(s_f + (kg * BM + row) * HC + 4 * ((col >> 2) ^ (row & (CH - 1)))) =
                f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the staged values are written
    barrier_no_fence();
#pragma unroll 2
    for (int it = tid; it < BM * HC / 8; it += 64 * NW * KG) {
      const int row = it / (HC / 8), c8 = it % (HC / 8);
      const int m = m0 + row, n = n0 + HC * part + 8 * c8;
      if (m >= g.M || n >= g.N) continue;  // N is a multiple of 8: a run is all in or all out
      f32x4 lo, hi;
#pragma unroll
      for (int k2 = 0; k2 < KG; ++k2) {
        const float* at = s_f + (k2 * BM + row) * HC;
        const f32x4 l2 = *(const f32x4*)(at + 4 * ((2 * c8) ^ (row & (CH - 1))));
        const f32x4 h2 = *(const f32x4*)(at + 4 * ((2 * c8 + 1) ^ (row & (CH - 1))));
        lo = k2 == 0 ? l2 : lo + l2;
        hi = k2 == 0 ? h2 : hi + h2;
      }
      float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      leave8<T>(g, slice, m, n, v);
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's reads of the staged rows are done
  }
}

template <typename T, bool AKC, bool BKC, typename C, bool TAIL>
__device__ __forceinline__ void any_product(const LinearProduct& g, int item, unsigned char* s_dyn) {
  const int tiles = ((g.M + C::BM - 1) / C::BM) * ((g.N + C::BN - 1) / C::BN);
  if (item / tiles * (int64_t)g.slice >= g.K) return;  // past the last slice: the grid may hold a few more
  tile_product<T, AKC, BKC, C, TAIL>(g, item % tiles, item / tiles, s_dyn);
}

// One workgroup per tile and slice: x W.
template <typename T, typename C, bool TAIL>
__global__ __launch_bounds__(kThreads, 2) void linear_fwd_kernel(LinearProduct g) {
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
    for (int p = w; p < c.n; p += kThreads / 64) v += c.part[(size_t)p * c.cols + col];
  s[w * 64 + l] = v;
  __syncthreads();
  if (w != 0 || col >= c.cols) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) v += s[i * 64 + l];
  store1((T*)c.out + col, v);
}

template <typename T, typename CX, typename CW, bool TAIL>
__global__ __launch_bounds__(kThreads, 2) void linear_bwd_kernel(LinearProduct gx, LinearProduct gw, ColumnSum sum,
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

// The tiles of moe_linear_plan.h.
using Tile0 = Tile<256, 256, 8, 2, 1, 2>;
using Tile1 = Tile<256, 128, 8, 4, 1, 3>;
using Tile2 = Tile<128, 128, 4, 2, 2, 2>;
using Tile3 = Tile<128, 64, 4, 2, 2, 3>;
// Four stages in flight for bf16; for fp32, whose stages take five times as long,
// two, so that two workgroups share a CU and one's prologue and epilogue run
// under the other's products (4330 x 1192 over 416: 65 -> 55 us).
template <typename T>
using Tile4 = Tile<64, 64, 4, 2, 2, sizeof(T) == 2 ? 4 : 2>;
// For a few rows: eight waves over the reduction, so that 512 k (fp32: 256) of it are
// on their way at once, and twice the CUs read the weights (bf16 in a captured
// graph: 8 x 768 -> 2048 5.5 -> 4.7 us, 1 x 2048 -> 768 9.2 -> 5.5; fp32 8 x 768 ->
// 2048 9.1 -> 7.3 us).
using Tile5 = Tile<32, 32, 1, 1, 8, 2>;

// The last plans of this thread by their sizes: a training or decoding loop asks
// for the same few shapes, and a search costs a few us of the host's time.
template <typename P, typename Fn>
const P& remembered(int T, int I, int O, int kind, Fn&& search) {
  struct Entry {
    int T, I, O, kind;
    P plan;
  };
  thread_local Entry entries[64] = {};
  const uint32_t h = ((uint32_t)T * 0x9e3779b1u) ^ ((uint32_t)I * 0x85ebca77u) ^ ((uint32_t)O * 0xc2b2ae3du) ^
                     ((uint32_t)kind * 0x27d4eb2fu);
  Entry& e = entries[(h >> 16) & 63];
  if (e.T != T || e.I != I || e.O != O || e.kind != kind) e = Entry{T, I, O, kind, search()};
  return e.plan;
}
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
  MOE_LAUNCH(kern, wide_grid(groups), dim3(kThreads), C::LDS, stream, g);
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
  MOE_LAUNCH(kern, wide_grid(p.x.groups + p.w.groups + sums), dim3(kThreads), lds, stream, gx, gw, sum,
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
  LinearProduct gx{T_, I, O, d, O, g.w, O, kActNone, nullptr, nullptr, dx_add, nullptr, dx, p.x.slice, nullptr};
  LinearProduct gw{I, O, T_, g.x, I, d, O, kActNone, nullptr, nullptr, nullptr, nullptr, dw, p.w.slice, nullptr};
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
  const LinearProduct p{g.T, g.O, g.I, g.x, g.I, g.w, g.O, g.act, bias, mul, residual, z, y, 0, nullptr};
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
