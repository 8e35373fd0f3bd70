// moe_adamw.hip -- an AdamW step over many tensors in one launch, with moments
// of 32 bits or of 8.
//
//   t = step + 1,  g' = grad_scale g
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr decay) - lr m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps)
//
// HBM-bound: every element of every tensor is read once and written once (22
// bytes of bf16 weight, gradient and 32-bit moments, 28 with an fp32 master, 10
// with 8-bit moments).
//
// What is held in fewer bits than it changes by is rounded up or down by a hash
// of the element's place, the step and the seed, up with the probability of what
// is left over: bf16 weights without a master (a step of 1e-5 beside a weight of
// 0.02 is a tenth of half a bf16 step: rounded to nearest it would never come
// about), and 8-bit moments (v moves by a thousandth of its distance to g^2, a
// sixtieth of a code's half step: to nearest it would stand still).  So the
// expected values are the exact ones, to 2^-12 of what a weight moves by and 2^-16
// of a code's step, but for v below its smallest code, which is raised to it.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "moe_common.h"
#include "moe_launch.h"
#include "moe_rows.h"

namespace moe {

namespace {

// ---- the hash ------------------------------------------------------------------

// Shifts and multiplications in turn; the multipliers here and in dithered() are three of the five 32-bit primes that the
// specification of the xxHash algorithm publishes.
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x85ebca77u;
  x = (x ^ (x >> 15)) * 0xc2b2ae3du;
  return x ^ (x >> 16);
}

// ---- moments in 8 bits ------------------------------------------------------------

// Blocks of 256 elements share a power-of-two scale.  m: E4M3 (bias 7, largest
// 448).  v, which has no sign and twice the range: 5 bits of exponent, 3 of
// mantissa, code c = (8 + c % 8) 2^(c / 8 - 34), 0 zero, 254 the largest, 1.75.
// Both keep NaN (0x7f, 255) for elements that are not finite (where v is not, m is
// not: g^2 does not leave the range of 64 bits).  A root of v that was rounded to
// zero would divide by eps alone: what is not zero stays so.
//
// m and v are formed in 64 bits, so that the code and the scale of every element
// are those of the formula: in 32 bits one in some millions would fall on the
// other side of a border, and differ by a whole code.
constexpr int kMaxM = 126, kMaxV = 254;

// The value of byte j of four codes of m, j a constant.
__device__ __forceinline__ float value_m(uint32_t codes, int j) {
  switch (j) {
    case 0: return __builtin_amdgcn_cvt_f32_fp8((int)codes, 0);
    case 1: return __builtin_amdgcn_cvt_f32_fp8((int)codes, 1);
    case 2: return __builtin_amdgcn_cvt_f32_fp8((int)codes, 2);
    default: return __builtin_amdgcn_cvt_f32_fp8((int)codes, 3);
  }
}
// The value of a code of v, whose bits are a double's but for the bias.  (255 need not read as NaN in a step: m's code
// says so too.)
__device__ __forceinline__ double value_v(uint32_t code) {
  return __hiloint2double(code == 0 ? 0 : (int)((code + ((1023 - 31) << 3)) << 17), 0);
}

// 2^e as a double.
__device__ __forceinline__ double pow2(int e) { return __hiloint2double((e + 1023) << 20, 0); }

// Exponent of the smallest power of two s with top <= 1.75 2^up s: 448 = 1.75 2^8.  By top's bits as fp32 (infinity,
// from a value past fp32's range, counts as the largest there).
__device__ __forceinline__ int scale_exponent(uint32_t bits, int up) {
  const int e = (int)(bits >> 23) - 127 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0) - up;
  return min(max(e, -126), 127);  // subnormal tops lie below the first
}

// Sign aside, the upper word of a double: 0x7ff00000 and more where it is not finite.
__device__ __forceinline__ uint32_t upper(double a) { return (uint32_t)__double2hiint(a) & 0x7fffffffu; }
__device__ __forceinline__ bool finite(double a) { return upper(a) < 0x7ff00000u; }

// Exponent and three bits of mantissa of the double (hi, lo), rounded up by an
// addition below them, 49 bits of h and a third: for the share (h + 1/3) / 2^16 of
// what is left over (the third keeps the border off values that short binary codes
// and gradients add up to).  Taken less e binades.  The lower words only carry.
__device__ __forceinline__ int eighths(int hi, uint32_t lo, uint32_t h, int e) {
  return (hi + (int)(h << 1) - (e << 20) + (lo > 0x55555555u ? 1 : 0)) >> 17;
}
// The code of m's size at the scale 2^e, where that is 8 (2^-6) or more.
__device__ __forceinline__ int size_code_m(double m, int e, uint32_t h) {
  return eighths((int)upper(m), (uint32_t)__double2loint(m), h, e) - ((1022 - 6) << 3);
}
// The same below: steps stay as large as there.  2^-6 is added, and its eight codes come off.
__device__ __forceinline__ int low_code_m(double m, int e, uint32_t h) {
  const double a = fma(fabs(m), pow2(-e), 0x1p-6);
  return eighths(__double2hiint(a), (uint32_t)__double2loint(a), h, 0) - ((1023 - 6) << 3);
}
__device__ __forceinline__ uint32_t code_m(double m, int size_code) {
  const uint32_t c = (uint32_t)min(size_code, kMaxM) | (((uint32_t)__double2hiint(m) >> 24) & 0x80u);
  return finite(m) ? c : 0x7fu;
}
// The code of v at the scale 2^e.
__device__ __forceinline__ uint32_t code_v(double v, int e, uint32_t h) {
  const int hi = __double2hiint(v);
  const int c = eighths(hi, (uint32_t)__double2loint(v), h, e) - ((1023 - 31) << 3);
  return v == 0.0 ? 0u : (uint32_t)min(max(c, 1), kMaxV);
}

// ---- the step ----------------------------------------------------------------------

struct AdamwArgs {
  const AdamwEntry* entries;
  const int64_t* starts;  // first chunk of each tensor, and their number behind the last
  int n;
  int64_t chunks;
  int32_t* counter;  // {steps done, workgroups done}
  const float* lr;
  const float* grad_scale;
  double beta1, beta2, log_beta1, log_beta2;
  float eps;
  uint32_t seed;
};

// Loads and stores of device memory through a pointer that was itself read from there (for the compiler it might point
// into LDS or scratch).
template <typename V>
__device__ __forceinline__ V get(const void* p) {
  return *(const __attribute__((address_space(1))) V*)p;
}
template <typename V>
__device__ __forceinline__ void put(void* p, V v) {
  *(__attribute__((address_space(1))) V*)p = v;
}

// Eight neighbouring elements, of which `live` are there (FULL: all).
template <bool FULL>
__device__ __forceinline__ void get8(const float* p, int live, float (&v)[8]) {
  if (FULL || live == 8) {
    const f32x4 lo = get<f32x4>(p), hi = get<f32x4>(p + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < 4 ? lo[j] : hi[j - 4];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < live ? get<float>(p + j) : 0.0f;
  }
}
template <bool FULL>
__device__ __forceinline__ void get8(const uint16_t* p, int live, float (&v)[8]) {
  if (FULL || live == 8) {
    const u32x4 q = get<u32x4>(p);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (j & 1) ? bf_hi(q[j >> 1]) : bf_lo(q[j >> 1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < live ? bf2f(get<uint16_t>(p + j)) : 0.0f;
  }
}
template <bool FULL>
__device__ __forceinline__ u32x2 get_codes(const void* p, int live) {
  if (FULL || live == 8) return get<u32x2>(p);
  u32x2 q = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j >> 2] |= (j < live ? (uint32_t)get<uint8_t>((const uint8_t*)p + j) : 0u) << (8 * (j & 3));
  return q;
}
template <bool FULL>
__device__ __forceinline__ void put8(float* p, int live, const float (&v)[8]) {
  if (FULL || live == 8) {
    put(p, f32x4{v[0], v[1], v[2], v[3]});
    put(p + 4, f32x4{v[4], v[5], v[6], v[7]});
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < live) put(p + j, v[j]);
  }
}
// bf16 values by their bits.
template <bool FULL>
__device__ __forceinline__ void put_bits(uint16_t* p, int live, const uint32_t (&q)[8]) {
  if (FULL || live == 8) {
    put(p, u32x4{q[0] | q[1] << 16, q[2] | q[3] << 16, q[4] | q[5] << 16, q[6] | q[7] << 16});
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < live) put(p + j, (uint16_t)q[j]);
  }
}
template <bool FULL>
__device__ __forceinline__ void put_codes(void* p, int live, u32x2 q) {
  if (FULL || live == 8) return put(p, q);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < live) put((uint8_t*)p + j, (uint8_t)(q[j >> 2] >> (8 * (j & 3))));
}

// A value that all lanes hold, in scalar registers.
template <typename V>
__device__ __forceinline__ V uniform(V v) {
  static_assert(sizeof(V) % 4 == 0, "whole words");
  uint32_t w[sizeof(V) / 4];
  __builtin_memcpy(w, &v, sizeof(V));
#pragma unroll
  for (size_t i = 0; i < sizeof(V) / 4; ++i) w[i] = __builtin_amdgcn_readfirstlane(w[i]);
  __builtin_memcpy(&v, w, sizeof(V));
  return v;
}

// What all elements share.
struct Shared {
  double gs;
  float step1, inv_root2, lr;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t key;
};

// What p goes down by but for the decay.  Root and reciprocal by the hardware's, each within 2^-23 of its value.
__device__ __forceinline__ float update(float m, float root, const Shared& sh, float eps) {
  return sh.step1 * (m * __builtin_amdgcn_rcpf(root * sh.inv_root2 + eps));
}
// The hardware's root of a subnormal is 0: what is near them is taken 2^100 times as large.
__device__ __forceinline__ float root_of(float v) {
  const bool tiny = v < 0x1p-100f;
  return __builtin_amdgcn_sqrtf(v * (tiny ? 0x1p100f : 1.0f)) * (tiny ? 0x1p-50f : 1.0f);
}
// Only where a wave has such a v: everywhere it costs a step with 32 bits 7 % (151M weights 802 -> 859 us), and one with
// 8 bits and its read-back 2 %, where the check would cost 4 (599, 611, 625).
__device__ __forceinline__ void update8(const float (&m)[8], const float (&v)[8], const Shared& sh, float eps,
                                        float (&u)[8]) {
  uint32_t least = 0xffffffffu;
#pragma unroll
  for (int j = 0; j < 8; ++j) least = min(least, __float_as_uint(v[j]) - 1);  // zeros count as large
  float root[8];
  if (__ballot(least < 0x0d800000u)) {  // 2^-100
#pragma unroll
    for (int j = 0; j < 8; ++j) root[j] = root_of(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) root[j] = __builtin_amdgcn_sqrtf(v[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = update(m[j], root[j], sh, eps);
}

// Where 1 - lr decay were taken as fp32 it would be a multiple of 2^-24, the same way for every element and step: a decay
// of 1e-7 came out as 1.15e-7, one of 1e-8 as none.  So p goes down by p (lr decay) + u in one rounding (an infinite one
// by u alone: infinity less itself would be NaN) ...
__device__ __forceinline__ float moved(float p, double decay, float u) {
  return p - (__builtin_isinf(p) ? u : fmaf(p, (float)decay, u));
}
// ... or, as bf16, up for the hash's share of what is left over: by an addition below the seven bits of mantissa, whose
// carry rounds up.  In 64 bits, as fp32 rounds to 2^-24 of p, where p may go down by less.  A share of 16 bits is up to
// as much off; where p moves by less than 2^-12 of itself, beside which that would count, it has 32.
__device__ __forceinline__ uint32_t dithered(float p, double decay, float u, uint32_t r) {
  const double to = fma((double)p, 1.0 - decay, -(double)u);
  const bool little = fabsf(fmaf(p, (float)decay, u)) < fabsf(p) * 0x1p-12f;
  const uint32_t h = (r * 0x9e3779b1u) & (little ? 0xffffffffu : 0xffff0000u);
  const uint64_t share = (uint64_t)h << 13;  // 52 - 7 - 32
  const uint64_t bits = ((uint64_t)__double_as_longlong(to) + share) >> 45 << 45;
  const uint32_t q = __float_as_uint((float)__longlong_as_double((long long)bits)) >> 16;
  return to != to ? 0x7fc0u : q;  // infinities stay: a share has none of their mantissa's bits
}
// Eight weights so.  fp32 and the upper 16 bits of the hash decide but where their sum is within four of a carry: fp32 is
// off by a step and a half (1 - decay, and the difference), the lower bits by one, for weights that keep half their
// size.  (One wave in sixteen has such a weight; 151M with 8-bit moments 352 -> 361 us, 385 with 64 bits everywhere;
// with 32-bit moments HBM hides it, 620.)
__device__ __forceinline__ void round8(const float (&p)[8], double decay, const float (&u)[8], const uint32_t (&r)[8],
                                       uint32_t (&q)[8]) {
  const float keep = (float)(1.0 - decay);
  bool close[8], any = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = fmaf(p[j], keep, -u[j]);
    const uint32_t sum = __float_as_uint(x) + ((r[j] * 0x9e3779b1u) >> 16);
    close[j] = (uint16_t)(sum + 4) < 8;
    any |= close[j];
    q[j] = x != x ? 0x7fc0u : sum >> 16;
  }
  if (__ballot(any)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = close[j] ? dithered(p[j], decay, u[j], r[j]) : q[j];
  }
}

// One pass over a chunk: eight elements a thread, from element `at` of tensor e on.
template <typename T, bool MASTER, bool SMALL, bool FULL>
__device__ __forceinline__ void adamw_pass(const AdamwArgs& g, const Shared& sh, const AdamwEntry& e, int64_t at) {
  const int live = FULL ? 8 : (int)min((int64_t)8, max((int64_t)0, e.numel - at));
  const double decay = (double)sh.lr * e.decay;
  float p[8], gr[8], u[8];
  get8<FULL>((const T*)e.grad + at, live, gr);
  if constexpr (MASTER) get8<FULL>(e.master + at, live, p);
  else get8<FULL>((const T*)e.param + at, live, p);
  uint32_t r[8];
  if (SMALL || (!MASTER && sizeof(T) == 2)) {
    const uint64_t place = (uint64_t)e.first * kAdamwBlock + (uint64_t)at;
    uint32_t key = sh.key;
    if (place >> 32) key ^= mix32((uint32_t)(place >> 32));
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = mix32(((uint32_t)place ^ key) ^ j);  // places of runs are multiples of 8
  }
  if constexpr (!SMALL) {
    const float b1 = (float)g.beta1, a1 = (float)(1.0 - g.beta1), b2 = (float)g.beta2, a2 = (float)(1.0 - g.beta2);
    const float gs = (float)sh.gs;
    float m[8], v[8];
    float *mp = (float*)e.m + at, *vp = (float*)e.v + at;
    get8<FULL>(mp, live, m);
    get8<FULL>(vp, live, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gj = gr[j] * gs;
      m[j] = b1 * m[j] + a1 * gj;
      v[j] = b2 * v[j] + a2 * gj * gj;
    }
    update8(m, v, sh, g.eps, u);
    put8<FULL>(mp, live, m);
    put8<FULL>(vp, live, v);
  } else {
    uint8_t *mp = (uint8_t*)e.m + at, *vp = (uint8_t*)e.v + at;
    const int64_t block = at / kAdamwBlock;
    const u32x2 mc = get_codes<FULL>(mp, live), vc = get_codes<FULL>(vp, live);
    // scales are powers of two: their products with the betas are exact
    const double bm = live > 0 ? g.beta1 * (double)get<float>(e.m_scale + block) : 0.0;
    const double bv = live > 0 ? g.beta2 * (double)get<float>(e.v_scale + block) : 0.0;
    const double am = (1.0 - g.beta1) * sh.gs, av = (1.0 - g.beta2) * sh.gs * sh.gs;
    double m[8], v[8];
    uint32_t top_m = 0, top_v = 0;  // as fp32 bits: the order of what is not negative
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double gj = (double)gr[j];
      m[j] = fma(gj, am, (double)value_m(mc[j >> 2], j & 3) * bm);
      v[j] = fma(gj * gj, av, value_v((vc[j >> 2] >> (8 * (j & 3))) & 255) * bv);
      const float mf = (float)m[j], vf = (float)v[j];
      u[j] = update(mf, root_of(vf), sh, g.eps);
      const bool ok = finite(m[j]);
      top_m = max(top_m, ok ? __float_as_uint(mf) & 0x7fffffffu : 0u);
      top_v = max(top_v, ok ? __float_as_uint(vf) : 0u);
    }
    top_m = row_max(top_m);  // the 32 lanes of a block
    top_v = row_max(top_v);
    top_m = max(top_m, (uint32_t)__shfl_xor((int)top_m, 16, kWave));
    top_v = max(top_v, (uint32_t)__shfl_xor((int)top_v, 16, kWave));
    const int em = scale_exponent(top_m, 8), ev = scale_exponent(top_v, 0);
    int c[8];
    bool low = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = size_code_m(m[j], em, r[j] & 0xffffu);
      low |= c[j] < 8;
    }
    if (__ballot(low)) {  // few waves: 2^-14.8 of the block's largest
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = c[j] < 8 ? low_code_m(m[j], em, r[j] & 0xffffu) : c[j];
    }
    u32x2 mq = {0, 0}, vq = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mq[j >> 2] |= code_m(m[j], c[j]) << (8 * (j & 3));
      const uint32_t cv = code_v(v[j], ev, r[j] >> 16);
      vq[j >> 2] |= (finite(m[j]) ? cv : 255u) << (8 * (j & 3));
    }
    put_codes<FULL>(mp, live, mq);
    put_codes<FULL>(vp, live, vq);
    if ((threadIdx.x & 31) == 0 && live > 0) {
      put(e.m_scale + block, (float)pow2(em));
      put(e.v_scale + block, (float)pow2(ev));
    }
  }
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = moved(p[j], decay, u[j]);
    put8<FULL>((float*)e.param + at, live, p);
  } else {
    uint32_t q[8];
    if constexpr (MASTER) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = moved(p[j], decay, u[j]);
        q[j] = f2bf(p[j]);
      }
    } else {
      round8(p, decay, u, r, q);
    }
    if constexpr (MASTER) put8<FULL>(e.master + at, live, p);
    put_bits<FULL>((uint16_t*)e.param + at, live, q);
  }
}

// The last of n tensors that begins at or before `chunk` (those before it are empty or done): 64 places are looked at
// at a time.
__device__ __forceinline__ int tensor_of(const int64_t* starts, int n, int64_t chunk) {
  int lo = 0;
  for (int left = n; left > 1;) {
    const int step = (left + 63) / 64, at = lane_id() * step;
    const bool before = at < left && get<int64_t>(starts + lo + at) <= chunk;
    const int last = max((int)__popcll(__ballot(before)) - 1, 0) * step;
    lo += last;
    left = min(step, left - last);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Workgroups of NT threads, of which every 256 take a chunk at a time.
template <typename T, bool MASTER, bool SMALL, int NT>
__global__ __launch_bounds__(NT, SMALL ? 4 : 1) void adamw_kernel(AdamwArgs g) {
  constexpr int AT_ONCE = NT / 256;  // chunks
  __shared__ Shared s_sh;
  const int tid = threadIdx.x;
  const int64_t begin = (int64_t)blockIdx.x * AT_ONCE + __builtin_amdgcn_readfirstlane(tid / 256);
  int i = 0;
  int64_t from = 0, to = 0;  // chunks of tensor i
  AdamwEntry e{};
  auto find = [&](int64_t chunk) {
    i += tensor_of(g.starts + i, g.n - i, chunk);
    from = uniform(g.starts[i]);
    to = uniform(g.starts[i + 1]);
    e = uniform(g.entries[i]);
  };
  if (begin < g.chunks) find(begin);
  if (tid == 0) {
    const int t = g.counter[0] + 1;
    const double lr = *g.lr;
    s_sh.gs = g.grad_scale != nullptr ? (double)*g.grad_scale : 1.0;
    s_sh.lr = (float)lr;
    s_sh.step1 = (float)(lr / -expm1(t * g.log_beta1));
    s_sh.inv_root2 = (float)(1.0 / sqrt(-expm1(t * g.log_beta2)));
    s_sh.key = mix32(mix32((uint32_t)t) + g.seed);
  }
  __syncthreads();
  const Shared sh = uniform(s_sh);
  for (int64_t chunk = begin; chunk < g.chunks; chunk += (int64_t)gridDim.x * AT_ONCE) {
    if (chunk >= to) find(chunk);
    const int64_t first = (chunk - from) * kAdamwChunk, at = first + 8 * (tid % 256);
    if (first + kAdamwChunk <= e.numel) adamw_pass<T, MASTER, SMALL, true>(g, sh, e, at);
    else adamw_pass<T, MASTER, SMALL, false>(g, sh, e, at);
  }
  // The last workgroup to get here counts the step: every one has read the counter.
  if (tid == 0 && (uint32_t)atomicAdd((uint32_t*)g.counter + 1, 1u) == gridDim.x - 1) {
    g.counter[1] = 0;
    g.counter[0] += 1;
  }
}

// The moments that codes stand for.  HBM-bound: 2 bytes read, 8 written an element.
__global__ __launch_bounds__(256) void adamw_moments_kernel(int64_t numel, const uint8_t* __restrict__ m,
                                                            const uint8_t* __restrict__ v,
                                                            const float* __restrict__ m_scale,
                                                            const float* __restrict__ v_scale, float* __restrict__ m_out,
                                                            float* __restrict__ v_out) {
  const int64_t at = ((int64_t)group_id() * 256 + threadIdx.x) * 8;
  if (at >= numel) return;
  const double ms = (double)m_scale[at / kAdamwBlock], vs = (double)v_scale[at / kAdamwBlock];
  const int live = (int)min((int64_t)8, numel - at);
  const u32x2 mc = get_codes<false>(m + at, live), vc = get_codes<false>(v + at, live);
  float a[8], b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t c = (vc[j >> 2] >> (8 * (j & 3))) & 255;
    a[j] = (float)((double)value_m(mc[j >> 2], j & 3) * ms);
    b[j] = c == 255 ? __builtin_nanf("") : (float)(value_v(c) * vs);
  }
  put8<false>(m_out + at, live, a);
  put8<false>(v_out + at, live, b);
}

struct Plan {
  uint32_t magic;
  int n, esize, small, master;
  int64_t chunks;
};
constexpr uint32_t kPlanMagic = 0x61646d77u;
constexpr size_t kPlanHead = 64;
static_assert(sizeof(Plan) <= kPlanHead, "the plan's head");

size_t starts_offset(int n) { return kPlanHead + (size_t)n * sizeof(AdamwEntry); }

}  // namespace

size_t adamw_plan_bytes(int n) { return starts_offset(n) + ((size_t)n + 1) * sizeof(int64_t); }

void adamw_make_plan(int n, const AdamwEntry* entries, int esize, bool small, bool master, void* plan) {
  Plan h{kPlanMagic, n, esize, small, master, 0};
  int64_t block = 0;
  for (int i = 0; i < n; ++i) {
    AdamwEntry e = entries[i];
    e.first = block;
    block += (e.numel + kAdamwBlock - 1) / kAdamwBlock;
    memcpy((char*)plan + kPlanHead + i * sizeof e, &e, sizeof e);
    memcpy((char*)plan + starts_offset(n) + i * sizeof(int64_t), &h.chunks, sizeof h.chunks);
    h.chunks += (e.numel + kAdamwChunk - 1) / kAdamwChunk;
  }
  memcpy((char*)plan + starts_offset(n) + n * sizeof(int64_t), &h.chunks, sizeof h.chunks);
  memset(plan, 0, kPlanHead);
  memcpy(plan, &h, sizeof h);
}

bool adamw_is_plan(const void* plan) {
  uint32_t magic;
  memcpy(&magic, plan, sizeof magic);
  return magic == kPlanMagic;
}

hipError_t launch_adamw(const void* plan, const void* plan_device, const AdamwStep& a, hipStream_t stream) {
  Plan h;
  memcpy(&h, plan, sizeof h);
  AdamwArgs g{};
  g.entries = (const AdamwEntry*)((const char*)plan_device + kPlanHead);
  g.starts = (const int64_t*)((const char*)plan_device + starts_offset(h.n));
  g.n = h.n;
  g.chunks = h.chunks;
  g.counter = a.counter;
  g.lr = a.lr;
  g.grad_scale = a.grad_scale;
  g.beta1 = a.beta1;
  g.beta2 = a.beta2;
  g.log_beta1 = a.beta1 > 0.0 ? log(a.beta1) : -__builtin_inf();
  g.log_beta2 = a.beta2 > 0.0 ? log(a.beta2) : -__builtin_inf();
  g.eps = (float)a.eps;
  g.seed = a.seed;
  auto run = [&](auto kernel, int threads, int most) {
    const int64_t groups = (h.chunks + threads / 256 - 1) / (threads / 256);
    const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>(groups, most)));
    MOE_LAUNCH(kernel, grid, dim3(threads), 0, stream, g);
    return hipGetLastError();
  };
  // 32-bit moments are bound by HBM, best with one small workgroup on a CU (151M weights with masters: 256 workgroups of
  // 256 threads 783 us or 5.4 TB/s, 512 827, 2048 840; 2M: 12.7, 14.8, 19.2, as workgroups queue up to say that they are
  // done).  The codes' arithmetic wants every SIMD full, by 256 workgroups of 1024 threads or, where the end counts for
  // little, 2048 of 256 (2M bf16 weights 10.7 and 17.5 us, 8M 26 and 33, 24M 64 either way, 32M 83.5 and 82, 151M 382 and
  // 358).
  constexpr int64_t kManyChunks = 16384;
  auto of = [&](auto t, auto master) {
    using T = decltype(t);
    constexpr bool MASTER = decltype(master)::value;
    if (!h.small) return run(adamw_kernel<T, MASTER, false, 256>, 256, 256);
    if (h.chunks >= kManyChunks) return run(adamw_kernel<T, MASTER, true, 256>, 256, 2048);
    return run(adamw_kernel<T, MASTER, true, 1024>, 1024, 256);
  };
  if (h.esize == 4) return of(0.0f, std::false_type{});
  return h.master ? of(uint16_t{}, std::true_type{}) : of(uint16_t{}, std::false_type{});
}

hipError_t launch_adamw_moments(int64_t numel, const uint8_t* m, const uint8_t* v, const float* m_scale,
                                const float* v_scale, float* m_out, float* v_out, hipStream_t stream) {
  MOE_LAUNCH(adamw_moments_kernel, wide_grid((numel + 2047) / 2048), dim3(256), 0, stream, numel, m, v, m_scale, v_scale,
             m_out, v_out);
  return hipGetLastError();
}

}  // namespace moe
