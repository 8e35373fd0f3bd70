// moe_route_scored.hip -- routing by softmax or sigmoid scores with a selection
// bias, expert groups and renormalised weights, and its backward.
//
//   s = softmax(l) or sigmoid(l),  c = s + bias,
//   group worth = sum of its 1 or 2 best c, the best groups stay,
//   idx = the k largest c (ties: lower index),  w = scale s_j [/ sum s_i].
#include "moe_common.h"
#include "moe_launch.h"

namespace moe {

namespace {

constexpr int kMaxGroups = 16;
constexpr int kRow = 16;  // lanes per token: a DPP row

struct RouteArgs {
  int T, E, k;
  int score;  // 0 softmax, 1 sigmoid
  int G, top_groups, group_top;
  int renorm;
  float scale;
  const float* logits;
  const float* bias;
  int32_t* idx;
  float* w;
  int per_lane;  // experts per lane, neighbours: ceil(E / 16)
  int on_lanes;  // every group is a whole number of lanes
};

template <int N>
__device__ __forceinline__ int ror(int v) { return __builtin_amdgcn_update_dpp(0, v, 0x120 + N, 0xf, 0xf, false); }
template <int N>
__device__ __forceinline__ float ror(float v) { return __int_as_float(ror<N>(__float_as_int(v))); }

// Over the 16 lanes of a token; every lane gets the same bits.
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, ror<8>(v));
  v = fmaxf(v, ror<4>(v));
  v = fmaxf(v, ror<2>(v));
  return fmaxf(v, ror<1>(v));
}
__device__ __forceinline__ float row_add(float v) {
  v += ror<8>(v);
  v += ror<4>(v);
  v += ror<2>(v);
  return v + ror<1>(v);
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, (uint32_t)ror<8>((int)v));
  v = max(v, (uint32_t)ror<4>((int)v));
  v = max(v, (uint32_t)ror<2>((int)v));
  return max(v, (uint32_t)ror<1>((int)v));
}

// Key whose order as an unsigned number is the order of a 64-bit value: -0
// equals +0, every NaN is the largest key, and no value has key 0.
__device__ __forceinline__ uint64_t order_key64(double v) {
  if (v != v) return ~0ull;
  const uint64_t u = (uint64_t)__double_as_longlong(v == 0.0 ? 0.0 : v);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

// The same for fp32 (NaN and the zeros aside), and back; -inf for keys at or below its.
constexpr uint32_t kKeyNegInf = 0x007fffffu;
__device__ __forceinline__ uint32_t order_key32(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  if (key <= kKeyNegInf) return -__builtin_inff();
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// The log of a score up to a term that every expert of the token shares (none
// for sigmoid): differences of these are exact where the scores underflow.
__device__ __forceinline__ float log_score(int score, float l) {
  if (score == 0) return l;
  return fminf(l, 0.0f) - log1pf(expf(-fabsf(l)));
}

// Renormalised weight of each lane's selected score (lanes `on`), the others 0:
// exp(a - max a) / sum over the token's 16 lanes, zeros where every selected score is zero.
__device__ __forceinline__ float renormalized(float a, bool on, bool poisoned) {
  const float m = row_max(on ? a : -__builtin_inff());
  float e = (on && m > -__builtin_inff()) ? expf(a - m) : 0.0f;
  if (poisoned || (on && a != a)) e = __builtin_nanf("");
  const float sum = row_add(e);
  return sum == 0.0f ? 0.0f : e / sum;
}

// Sorts v descending (Batcher's odd-even merge sort; N a power of two).
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t hi = max(v[i + j], v[i + j + q]), lo = min(v[i + j], v[i + j + q]);
            v[i + j] = hi;
            v[i + j + q] = lo;
          }
}

template <int V>
struct RouteLds {
  uint64_t value[4][4][kRow * V];  // wave, token of the wave, expert
  int32_t sel[4][4][kRow];
  float group[4][4][kMaxGroups];
};

__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // the wave's LDS writes before its reads
}

__device__ __forceinline__ double as_double(uint64_t u) { return __longlong_as_double((long long)u); }

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// The choice of one token in 64 bits by the whole wave, whatever its logits hold:
// fills sel, uses `value`, returns whether the token has no scores (softmax with
// a NaN or +inf).  For the few tokens that fp32 cannot decide; lane l holds the
// experts l + 64 i.
__device__ __forceinline__ bool choose_exactly(const RouteArgs& g, const float* lt, uint64_t* value, int32_t* sel) {
  constexpr int P = kMaxExperts / kWave;
  const double inf = __builtin_inf();
  const int lane = threadIdx.x & 63;
  double l[P], c[P], m = -inf;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + kWave * i;
    l[i] = e < g.E ? (double)lt[e] : -inf;
    bad |= !(l[i] < inf);
    m = fmax(m, l[i]);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmax(m, __shfl_xor(m, o, kWave));
  const bool poisoned = g.score == 0 && __ballot(bad) != 0;
  const bool two = g.G > 1 && g.group_top == 2;
  if (g.bias != nullptr || two) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      c[i] = l[i] == -inf ? 0.0 : exp(g.score == 0 ? l[i] - m : -l[i]);
      sum += c[i];
    }
    if (g.score == 0) sum = wave_sum64(sum);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = lane + kWave * i;
      c[i] = g.score == 0 ? c[i] / (sum > 0.0 ? sum : 1.0) : 1.0 / (1.0 + c[i]);
      if (poisoned) c[i] = __builtin_nan("");
      if (g.bias != nullptr) c[i] += (double)g.bias[min(e, g.E - 1)];
      if (l[i] == -inf) c[i] = -inf;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) c[i] = l[i];
  }
  uint32_t kept = 0xffffu;
  const int size = g.E / g.G;
  if (g.G > 1) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + kWave * i < g.E) value[lane + kWave * i] = (uint64_t)__double_as_longlong(c[i]);
    wave_lds_order();
    // four lanes per group
    const int grp = lane & 15;
    double a = -inf, b = -inf;
    bool nan = false;
    if (grp < g.G)
#pragma unroll 2
      for (int j = lane >> 4; j < size; j += 4) {
        const double v = as_double(value[grp * size + j]);
        nan |= v != v;
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
#pragma unroll
    for (int o = 16; o <= 32; o *= 2) {
      const double a2 = __shfl_xor(a, o, kWave), b2 = __shfl_xor(b, o, kWave);
      b = fmax(fmin(a, a2), fmax(b, b2));
      a = fmax(a, a2);
      nan |= __shfl_xor((int)nan, o, kWave) != 0;
    }
    const uint64_t worth = order_key64(nan ? __builtin_nan("") : (two && b > -inf ? a + b : a));
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < g.G; ++j) {
      const uint64_t o = __shfl(worth, j, kRow);
      rank += (o > worth || (o == worth && j < grp)) ? 1 : 0;
    }
    kept = (uint32_t)__ballot(grp < g.G && rank < g.top_groups) & 0xffffu;
  }
  uint64_t key[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + kWave * i;
    // without a bias the logits' own order, which rounding of the scores cannot blur
    const double by = g.bias == nullptr ? l[i] : c[i];
    key[i] = e < g.E ? order_key64((kept >> (e / size)) & 1 ? by : -inf) : 0;
  }
  for (int r = 0; r < g.k; ++r) {
    uint64_t best = key[0];
    int at = lane;
#pragma unroll
    for (int i = 1; i < P; ++i)
      if (key[i] > best) {
        best = key[i];
        at = lane + kWave * i;
      }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const uint64_t ob = __shfl_xor(best, o, kWave);
      const int oe = __shfl_xor(at, o, kWave);
      if (ob > best || (ob == best && oe < at)) {
        best = ob;
        at = oe;
      }
    }
    if (lane == 0) sel[r] = at;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (at == lane + kWave * i) key[i] = 0;
  }
  return poisoned;
}

// Sixteen lanes per token, four tokens per wave; lane i of a token holds the
// per_lane experts from per_lane i on in V registers (FULL: all of them, E = 16 V).
//
// The work is VALU instructions, not bytes (a token's logits are read once): a
// sort of V keys per lane, then k + 1 rounds of a maximum over 16 lanes.  So choice
// scores are formed in fp32 and packed into 32-bit keys, the order key with its
// low four bits given to the expert's place in its lane: sorting is min and
// max, a round a DPP row maximum, after which the winner's lane moves up.  A
// key is off by at most 2^-19 of its value, the scores by a few 2^-24 (below).
// Where two neighbours of the sorted k + 1 best are nearer than that, the 16
// best are ordered by their 64-bit choice scores; where that does not settle
// it, or a group is in doubt, or a value is not finite, the wave decides that
// token over all experts in 64 bits (choose_exactly).  The choice is the exact one on every path.
//
// Measured at 16384 tokens: softmax over 128 experts 5.8 us, sigmoid with a bias
// over 256 10.1 us, in 8 groups of which 4 are kept 13.3 us (everything in 64
// bits, a wave per token: 149 us; the 17.8 MB alone would take 3.6 us).  Logits
// with many equal values take the exact ways more often: 18 us on a grid of a
// quarter.
template <int V, bool FULL>
__global__ __launch_bounds__(256) void route_scored_kernel(RouteArgs g) {
  __shared__ RouteLds<V> s;
  const float inf = __builtin_inff();
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, tok = lane >> 4, li = lane & 15;
  const int64_t t = (int64_t)group_id() * 16 + 4 * wv + tok;
  const bool live = t < g.T;
  const float* lt = g.logits + (live ? t : g.T - 1) * g.E;
  const int E = FULL ? kRow * V : g.E, k = g.k, per_lane = FULL ? V : g.per_lane;
  const int e0 = li * per_lane, n = FULL ? V : min(max(E - e0, 0), per_lane);  // this lane's experts
  int32_t* sel = s.sel[wv][tok];
  // V neighbours from p + e0; past the lane's experts any value of the row
  auto fetch = [&](const float* p, float (&v)[V]) {
    if (FULL && V >= 4) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const f32x4 q = *(const f32x4*)(p + e0 + i);
#pragma unroll
        for (int j = 0; j < 4 && i + j < V; ++j) v[i + j] = q[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = p[FULL ? e0 + i : min(e0 + i, E - 1)];
    }
  };
  float c[V];
  fetch(lt, c);
  if (!FULL)
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = i < n ? c[i] : -inf;
  // scores only where a bias or a sum meets them, or the weights need their sum
  const bool by_score = g.bias != nullptr || (g.G > 1 && g.group_top == 2);
  float top = 0.0f, sum = 1.0f, slack = 1e-30f;
  if (g.score == 0 && (by_score || !g.renorm)) {
    float m = c[0], ex[V];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, c[i]);
    top = row_max(m);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ex[i] = quick_exp(c[i] - top);  // a row of -inf: NaN, which goes the exact way
      sum += ex[i];
    }
    sum = row_add(sum);
    if (by_score) {
      const float inv = __builtin_amdgcn_rcpf(sum);
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = c[i] == -inf ? -inf : ex[i] * inv;
      // |error| of a softmax score: (2.5 |d| + 40) 2^-24 s, d its logit's distance from the largest
      // (argument and result of exp, the sum of E terms, the quotient), so at most 2.5 2^-20 of
      // the largest score 1 / sum; twice that between two
      slack += inv * 0x1p-17f;
    }
  } else if (by_score) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = c[i] == -inf ? -inf : __builtin_amdgcn_rcpf(1.0f + quick_exp(-c[i]));
    slack += 0x1p-20f;  // |error| of a sigmoid: at most 5 2^-24
  }
  if (g.bias != nullptr) {
    float b[V];
    fetch(g.bias, b);
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = c[i] == -inf ? -inf : c[i] + b[i];
  }
  bool exactly = false;  // fp32 cannot decide
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    exactly |= (FULL || i < n) && __builtin_amdgcn_classf(c[i], 0x203);  // NaN or +inf
    key[i] = FULL || i < n ? (order_key32(c[i]) & ~15u) | (uint32_t)(15 - i) : 0u;
  }
  sort_down(key);
  // whether one key's value surely lies above another's
  auto apart = [&](float hi, float lo) {
    return hi - lo > 1.25f * 0x1p-19f * fmaxf(fabsf(hi), lo > -inf ? fabsf(lo) : 0.0f) + slack;
  };
  if (g.G > 1) {
    float a, b = -inf;
    const int lpg = kRow / g.G;  // lanes per group, where groups are whole lanes
    const int size = E / g.G;
    if (g.on_lanes) {
      a = c[0];
#pragma unroll
      for (int i = 1; i < V; ++i) {
        b = __builtin_amdgcn_fmed3f(a, b, c[i]);
        a = fmaxf(a, c[i]);
      }
      for (int o = 1; o < lpg; o <<= 1) {
        const float a2 = __shfl_xor(a, o, kRow), b2 = __shfl_xor(b, o, kRow);
        b = fmaxf(fminf(a, a2), fmaxf(b, b2));
        a = fmaxf(a, a2);
      }
    } else {
      float* cs = (float*)s.value[wv][tok];
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) cs[e0 + i] = c[i];
      wave_lds_order();
      a = -inf;
      if (li < g.G)
        for (int j = 0; j < size; ++j) {
          const float v = cs[li * size + j];
          b = fmaxf(b, fminf(a, v));
          a = fmaxf(a, v);
        }
    }
    const bool two = g.group_top == 2 && b > -inf;
    const float worth = two ? a + b : a;
    const float size_of = a > -inf ? fabsf(a) + (two ? fabsf(b) : 0.0f) : 0.0f;
    // two scores each, and the roundings of two sums with the bias and of their sum
    const float near = by_score ? 2.0f * slack + 0x1p-21f * row_max(size_of) : 0.0f;
    const bool has = g.on_lanes || li < g.G;
    if (g.on_lanes ? (li & (lpg - 1)) == 0 : has) s.group[wv][tok][g.on_lanes ? li / lpg : li] = worth;
    wave_lds_order();
    int above = 0, not_below = 0;  // groups surely above this lane's, and those not surely below
    const int own = g.on_lanes ? li / lpg : li;
    for (int j = 0; j < g.G; ++j) {
      const float o = s.group[wv][tok][j];
      if (j == own) continue;
      if (by_score) {
        above += o > worth + near ? 1 : 0;
        not_below += o < worth - near ? 0 : 1;
      } else {
        const int is = o > worth || (o == worth && j < own) ? 1 : 0;
        above += is;
        not_below += is;
      }
    }
    bool keep = above < g.top_groups;
    const bool doubt = has && keep != (not_below < g.top_groups);
    if (V > 1 && g.on_lanes && g.score == 1) {
      if (__ballot(doubt)) {
        // the worths again from 64-bit scores of each lane's two best
        double best[2];
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          const uint32_t q = j ? key[1] : key[0];
          const int e = e0 + 15 - (int)(q & 15u);
          const double v = 1.0 / (1.0 + exp(-(double)lt[e])) + (g.bias != nullptr ? (double)g.bias[e] : 0.0);
          best[j] = q > kKeyNegInf ? v : -__builtin_inf();
        }
        // the third best may be the second in truth
        if (V > 2 && !apart(key_value(key[1] & ~15u), key_value(key[V > 2 ? 2 : 0] & ~15u))) exactly = true;
        double a2 = fmax(best[0], best[1]), b2 = fmin(best[0], best[1]);
        for (int o = 1; o < lpg; o <<= 1) {
          const double a3 = __shfl_xor(a2, o, kRow), b3 = __shfl_xor(b2, o, kRow);
          b2 = fmax(fmin(a2, a3), fmax(b2, b3));
          a2 = fmax(a2, a3);
        }
        const uint64_t worth2 = order_key64(g.group_top == 2 && b2 > -__builtin_inf() ? a2 + b2 : a2);
        int rank = 0;
        for (int j = 0; j < g.G; ++j) {
          const uint64_t o = __shfl(worth2, j * lpg, kRow);
          rank += (o > worth2 || (o == worth2 && j < own)) ? 1 : 0;
        }
        keep = rank < g.top_groups;
      }
    } else {
      exactly |= doubt;
    }
    if (g.on_lanes) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = keep ? key[i] : (kKeyNegInf & ~15u) | (uint32_t)(15 - i);
    } else {
      const uint32_t kept = (uint32_t)(__ballot(has && keep) >> (kRow * tok)) & 0xffffu;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int at = e0 + 15 - (int)(key[i] & 15u);
        if (key[i] != 0 && !((kept >> (at / size)) & 1)) key[i] = (kKeyNegInf & ~15u) | (key[i] & 15u);
      }
      sort_down(key);
    }
  }
  // the best in turn: lane r keeps the r-th; equal keys: the lower lane
  uint32_t mine = 0, last = 0;
  auto next_best = [&](int r) {
    last = row_max(key[0]);
    const uint64_t same = __ballot(key[0] == last);
    const uint32_t row = (uint32_t)(same >> (kRow * tok)) & 0xffffu;
    const bool won = li == __ffs(row) - 1;
    if (won && r < kRow) sel[r] = e0 + 15 - (int)(last & 15u);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = won ? (i + 1 < V ? key[i + 1] : 0u) : key[i];
    mine = li == r ? last : mine;
  };
  const int rounds = k < E ? k + 1 : k;
  for (int r = 0; r < rounds; ++r) next_best(r);
  bool close = false;
  {
    const float v = key_value(mine & ~15u);
    uint32_t after = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mine, 0x101, 0xf, 0xf, false);  // lane li + 1's
    if (li == kRow - 1) after = last;                                                             // k = 16
    const bool pair = li < k - 1 || (li == k - 1 && k < E);
    close = pair && !apart(v, key_value(after & ~15u));
    exactly |= li < k && !(v > -inf);  // an unavailable expert is listed
  }
  const bool few = k < kRow && (g.score == 1 || g.bias == nullptr);  // the 16 best can settle it
  exactly |= close && !few;
  bool poisoned = false;
  if (__ballot(close || exactly)) {
    const uint64_t ties = __ballot(close);
    if (few && ties) {
      // the 16 best (all of them, where E <= 16) by 64-bit choice scores
      const int cand = min(E, kRow);
      for (int r = rounds; r < cand; ++r) next_best(r);
      const float v = key_value(mine & ~15u);
      const bool settled = E <= kRow || apart(__shfl(v, k - 1, kRow), __shfl(v, kRow - 1, kRow));
      exactly |= ((ties >> (kRow * tok)) & 0xffffu) != 0 && !settled;
      wave_lds_order();
      const int e = li < cand ? sel[li] : 0;
      const float le = lt[e];
      double by = (double)le;
      if (g.bias != nullptr) by = 1.0 / (1.0 + exp(-by)) + (double)g.bias[e];
      const uint64_t rank_by = li < cand ? order_key64(v > -inf ? by : -__builtin_inf()) : 0;
      int rank = 0;
      for (int j = 0; j < cand; ++j) {
        const uint64_t o = __shfl(rank_by, j, kRow);
        const int oe = __shfl(e, j, kRow);
        rank += (o > rank_by || (o == rank_by && oe < e)) ? 1 : 0;
      }
      wave_lds_order();
      if (li < cand && rank < k) sel[rank] = e;
    }
    const uint64_t open = __ballot(exactly);
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      if (((open >> (kRow * q)) & 0xffffu) == 0) continue;
      const int64_t tq = min((int64_t)group_id() * 16 + 4 * wv + q, (int64_t)g.T - 1);
      const bool none = choose_exactly(g, g.logits + tq * g.E, s.value[wv][q], s.sel[wv][q]);
      if (q == tok) poisoned = none;
    }
  }
  wave_lds_order();
  const bool on = li < k;
  const int e = on ? sel[li] : 0;
  const float le = lt[e];
  float we;
  if (g.renorm) {
    we = renormalized(log_score(g.score, le), on, poisoned);
  } else if (g.score == 0) {
    we = poisoned ? __builtin_nanf("") : (le > -inf ? expf(le - top) / sum : 0.0f);
  } else {
    we = 1.0f / (1.0f + expf(-le));
  }
  if (live && on) {
    g.idx[t * k + li] = e;
    g.w[t * k + li] = g.scale * we;
  }
}

// The backward: sixteen lanes per token as in the forward.  Lanes j < k hold the
// selected pairs' terms (an index listed twice: each holds the sum of its
// terms), which go through an LDS row of zeros so that every lane writes whole
// runs of the token's dlogits once.
//
// A confident router's gradient is a small difference: of 1 and a score, of g
// and its mean over weights of which one is nearly 1.  None is formed from
// rounded values that near each other: 1 - s of a sigmoid is 1 / (1 + exp(l)),
// and as the weights sum to 1
//   g_j - sum_i p_i g_i = sum_i p_i (g_j - g_i),
// plain softmax alike over all experts, g = 0 where not selected:
//   g_e - sum_i s_i g_i = sum_{i selected} s_i (g_e - g_i) + g_e sum_{i not selected} s_i.
//
// HBM-bound: the output, and for plain softmax (DENSE, the only one whose
// gradient reaches every expert) the logits.  QUAD: runs of four experts, every
// sixteenth run of a lane; otherwise single experts.  A call at 16384 tokens,
// plain softmax: 128 experts 7.1 us, 256 8.6 us (with 1 - s and g - sum p g as
// differences of rounded values 7.1 and 8.2 us, and no correct digit left
// where a score is within 2^-24 of 1).
template <bool QUAD, bool DENSE>
__global__ __launch_bounds__(256) void route_scored_bwd_kernel(int T, int E, int k, int score, int renorm, float scale,
                                                               const float* __restrict__ logits,
                                                               const int32_t* __restrict__ idx,
                                                               const float* __restrict__ dg, float* __restrict__ dl) {
  constexpr int R = QUAD ? 4 : 1, N = kMaxExperts / (kRow * R);  // experts per run, runs per lane
  __shared__ __attribute__((aligned(16))) float s_d[4][4][kMaxExperts];
  const float inf = __builtin_inff();
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, tok = lane >> 4, li = lane & 15;
  const int64_t row = (int64_t)group_id() * 16 + 4 * wv + tok;
  const bool live = row < T;
  const int64_t t = live ? row : T - 1;
  const float* lt = logits + t * E;
  float* d_row = s_d[wv][tok];
  int e_l = -1;
  float g = 0.0f, a = -inf;
  if (li < k) {
    const int e = idx[t * k + li];
    if (e >= 0 && e < E) {
      e_l = e;
      g = dg[t * k + li];
      a = lt[e];
    }
  }
  float l[N][R];
  float m = -inf, sum = 1.0f;
  if (DENSE) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = R * (li + kRow * i);
      if (QUAD) {
        const f32x4 q = e < E ? *(const f32x4*)(lt + e) : f32x4{-inf, -inf, -inf, -inf};
#pragma unroll
        for (int j = 0; j < R; ++j) l[i][j] = q[j];
      } else {
        l[i][0] = e < E ? lt[e] : -inf;
      }
#pragma unroll
      for (int j = 0; j < R; ++j) {
        nan |= l[i][j] != l[i][j];
        m = fmaxf(m, l[i][j]);
      }
    }
    m = row_max(m);
    if ((__ballot(nan) >> (kRow * tok)) & 0xffff) m = __builtin_nanf("");
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) {
        l[i][j] = l[i][j] == -inf ? 0.0f : quick_exp(l[i][j] - m);  // NaN where the row is
        sum += l[i][j];
      }
    sum = row_add(sum);
  }
  const bool avail = e_l >= 0 && a != -inf;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = R * (li + kRow * i);
    if (QUAD) *(f32x4*)(d_row + e) = f32x4{0.f, 0.f, 0.f, 0.f};
    else d_row[e] = 0.0f;
  }
  // sum_i p_i (g - g_i) over the token's lanes, from each lane's own p and g
  auto spread = [&](float p, float g_own) {
    float p_i = p, g_i = g_own, v = 0.0f;
#pragma unroll
    for (int i = 1; i < kRow; ++i) {
      p_i = ror<1>(p_i);
      g_i = ror<1>(g_i);
      v += p_i * (g_own - g_i);
    }
    return v;
  };
  if (!avail) g = 0.0f;
  float d, sg = 0.0f;  // DENSE: sg = sum_i s_i g_i
  if (DENSE) {
    // marks the selected experts, leaves l only to the others, and adds those
    wave_lds_order();
    if (e_l >= 0) d_row[e_l] = (float)(li + 1);
    wave_lds_order();
    float others = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = R * (li + kRow * i);
      f32x4 mark;
      if (QUAD) mark = *(const f32x4*)(d_row + e);
      else mark[0] = d_row[e];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        l[i][j] = mark[j] == 0.0f ? l[i][j] : 0.0f;
        others += l[i][j];
      }
    }
    others = row_add(others) / sum;
    const float se = avail ? expf(a - m) / sum : 0.0f;
    sg = row_add(se * g);
    float g_e = g, listed = 1.0f;
    if (__ballot(e_l >= 0 && d_row[max(e_l, 0)] != (float)(li + 1))) {
      // an index listed twice: the sum of its g, its score shared out among the listings
      float g_i = g;
      int e_i = e_l;
#pragma unroll 1
      for (int i = 1; i < kRow; ++i) {
        e_i = ror<1>(e_i);
        g_i = ror<1>(g_i);
        g_e += e_i == e_l ? g_i : 0.0f;
        listed += e_i == e_l ? 1.0f : 0.0f;
      }
    }
    d = scale * se * (spread(se / listed, g_e) + g_e * others);
  } else {
    const float s_not = score == 0 ? 1.0f : 1.0f / (1.0f + expf(a));  // 1 - s
    if (renorm) {
      const float p = renormalized(log_score(score, a), e_l >= 0, false);
      d = scale * p * spread(p, g) * s_not;
    } else {
      d = scale * g * s_not / (1.0f + expf(-a));
    }
  }
  if (!avail) d = 0.0f;
  float total = d;
  if (!DENSE) {
    total = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int ej = __shfl(e_l, j, kRow);
      const float dj = __shfl(d, j, kRow);
      total += ej == e_l ? dj : 0.0f;
    }
  }
  wave_lds_order();
  if (e_l >= 0) d_row[e_l] = total;
  wave_lds_order();
  const float back = DENSE && sum > 0.0f ? -scale * sg / sum : (sum != sum ? sum : 0.0f);
  float* out = dl + t * E;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = R * (li + kRow * i);
    if (e >= E || !live) continue;
    if (QUAD) {
      f32x4 q = *(const f32x4*)(d_row + e);
      if (DENSE)
#pragma unroll
        for (int j = 0; j < R; ++j) q[j] += back * l[i][j];
      *(f32x4*)(out + e) = q;
    } else {
      out[e] = DENSE ? d_row[e] + back * l[i][0] : d_row[e];
    }
  }
}

template <int V>
hipError_t route_launch(const RouteArgs& g, bool aligned, hipStream_t stream) {
  const dim3 grid = wide_grid(((int64_t)g.T + 15) / 16), block(256);
  if (aligned && g.E == kRow * V) MOE_LAUNCH((route_scored_kernel<V, true>), grid, block, 0, stream, g);
  else MOE_LAUNCH((route_scored_kernel<V, false>), grid, block, 0, stream, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_scored(int T, int E, int k, int score, int n_groups, int top_groups, int group_top,
                               bool renormalize, float scale, const float* logits, const float* bias, int32_t* idx,
                               float* w, hipStream_t stream) {
  RouteArgs g{T, E, k, score, n_groups, top_groups, group_top, (int)renormalize, scale, logits, bias, idx, w, 0, 0};
  g.per_lane = (E + kRow - 1) / kRow;
  g.on_lanes = E % kRow == 0 && kRow % n_groups == 0;
  const bool aligned = (((uintptr_t)logits | (uintptr_t)bias) & 15) == 0;
  switch (g.per_lane) {
    case 1: return route_launch<1>(g, aligned, stream);
    case 2: return route_launch<2>(g, aligned, stream);
    case 3: case 4: return route_launch<4>(g, aligned, stream);
    case 5: case 6: case 7: case 8: return route_launch<8>(g, aligned, stream);
    default: return route_launch<16>(g, aligned, stream);
  }
}

hipError_t launch_route_scored_bwd(int T, int E, int k, int score, bool renormalize, float scale, const float* logits,
                                   const int32_t* idx, const float* dg, float* dlogits, hipStream_t stream) {
  const dim3 grid = wide_grid(((int64_t)T + 15) / 16), block(256);
  const bool quad = E % 4 == 0 && (((uintptr_t)logits | (uintptr_t)dlogits) & 15) == 0;
  auto run = [&](auto kernel) {
    MOE_LAUNCH(kernel, grid, block, 0, stream, T, E, k, score, (int)renormalize, scale, logits, idx, dg, dlogits);
    return hipGetLastError();
  };
  if (score == 0 && !renormalize)
    return quad ? run(route_scored_bwd_kernel<true, true>) : run(route_scored_bwd_kernel<false, true>);
  return quad ? run(route_scored_bwd_kernel<true, false>) : run(route_scored_bwd_kernel<false, false>);
}

}  // namespace moe
