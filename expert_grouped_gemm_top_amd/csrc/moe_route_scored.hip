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
  int quads;     // per_lane and E are multiples of 4 and the rows 16-byte aligned
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

// Sorts v descending (a bitonic network; N a power of two).
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&v)[N]) {
#pragma unroll
  for (int size = 2; size <= N; size *= 2)
#pragma unroll
    for (int stride = size / 2; stride > 0; stride /= 2)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int j = i ^ stride;
        if (j > i) {
          const uint32_t hi = max(v[i], v[j]), lo = min(v[i], v[j]);
          const bool down = (i & size) == 0;
          v[i] = down ? hi : lo;
          v[j] = down ? lo : hi;
        }
      }
}

template <int V>
struct RouteLds {
  double value[4][4][kRow * V];  // wave, token of the wave, expert: what groups are weighed by
  int32_t sel[4][4][kRow];
  float group[4][4][kMaxGroups];
};

__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // the wave's LDS writes before its reads
}

__device__ __forceinline__ double row_max(double v) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) v = fmax(v, __shfl_xor(v, o, kRow));
  return v;
}

// The choice of the wave's four tokens in 64 bits, whatever their logits hold;
// fills sel.  For the rare wave whose fp32 choice scores are too close to tell.
template <int V>
__device__ void choose_exactly(const RouteArgs& g, const float* lt, int wv, int tok, int li, RouteLds<V>& s) {
  const int E = g.E, e0 = li * g.per_lane;
  float l[V];
  double sc[V];
  double m = -__builtin_inf();
  bool nan = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = e0 + i;
    l[i] = i < g.per_lane && e < E ? lt[e] : -__builtin_inff();
    nan |= l[i] != l[i];
    m = fmax(m, (double)l[i]);
  }
  m = row_max(m);
  const bool poisoned = g.score == 0 && (((__ballot(nan) >> (kRow * tok)) & 0xffff) != 0 || m == __builtin_inf());
  double sum = 0.0;
  for (int i = 0; i < V; ++i) {
    if (g.score == 0) sc[i] = l[i] > -__builtin_inff() ? exp((double)l[i] - m) : 0.0;
    else sc[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    sum += sc[i];
  }
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, kRow);
  uint64_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = e0 + i;
    key[i] = 0;
    if (i >= g.per_lane || e >= E) continue;
    if (g.score == 0) sc[i] = poisoned ? __builtin_nan("") : (sum > 0.0 ? sc[i] / sum : 0.0);
    const double c = l[i] == -__builtin_inff() ? -__builtin_inf() : sc[i] + (g.bias != nullptr ? (double)g.bias[e] : 0.0);
    // without a bias the logits' own order, which rounding of the scores cannot blur
    const double by = g.bias != nullptr ? c : (double)l[i];
    key[i] = order_key64(by);
    s.value[wv][tok][e] = g.group_top == 1 ? by : c;
  }
  if (g.G > 1) {
    wave_lds_order();
    const int size = E / g.G;
    uint64_t worth = 0;
    if (li < g.G) {
      double a = -__builtin_inf(), b = -__builtin_inf();
      bool bad = false;
      for (int j = 0; j < size; ++j) {
        const double v = s.value[wv][tok][li * size + j];
        bad |= v != v;
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
      worth = order_key64(bad ? __builtin_nan("") : (g.group_top == 2 && b > -__builtin_inf() ? a + b : a));
    }
    int rank = 0;
    for (int j = 0; j < g.G; ++j) {
      const uint64_t o = __shfl(worth, j, kRow);
      rank += (o > worth || (o == worth && j < li)) ? 1 : 0;
    }
    const uint32_t kept = (uint32_t)(__ballot(li < g.G && rank < g.top_groups) >> (kRow * tok)) & 0xffffu;
    const uint64_t out = order_key64(-__builtin_inf());
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] != 0 && !((kept >> ((e0 + i) / size)) & 1)) key[i] = out;
  }
  for (int r = 0; r < g.k; ++r) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    int e = e0 + at;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) {
      const uint64_t ob = __shfl_xor(best, o, kRow);
      const int oe = __shfl_xor(e, o, kRow);
      if (ob > best || (ob == best && oe < e)) {
        best = ob;
        e = oe;
      }
    }
    if (li == 0) s.sel[wv][tok][r] = e;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i == e) key[i] = 0;
  }
}

// Sixteen lanes per token, four tokens per wave; lane i of a token holds the
// per_lane experts from per_lane i on, V >= per_lane registers.
//
// Choice scores are formed in fp32 and packed into 32-bit keys: the order key
// with its low four bits given to the expert's place in its lane, so that
// sorting a lane's keys is min and max, and the lanes' best is a maximum over a DPP row; each
// round the winner's lane moves up.  Such a key is off by at most 2^-19 of the
// value, the scores by a few 2^-24 (below); where two neighbours of the sorted k + 1 best, or
// the last kept and the first dropped group, are nearer than those errors reach, or any value is not finite, the wave decides
// in 64 bits instead (choose_exactly).  So the choice is always the exact one.
template <int V>
__global__ __launch_bounds__(256) void route_scored_kernel(RouteArgs g) {
  __shared__ RouteLds<V> s;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, tok = lane >> 4, li = lane & 15;
  const int64_t t = (int64_t)blockIdx.x * 16 + 4 * wv + tok;
  const bool live = t < g.T;
  const float* lt = g.logits + (live ? t : g.T - 1) * g.E;
  const int E = g.E, k = g.k, e0 = li * g.per_lane;
  float l[V];
  if (V >= 4 && g.quads) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const bool in = i < g.per_lane && e0 + i < E;
      const f32x4 q = in ? *(const f32x4*)(lt + e0 + i) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < V) l[i + j] = in ? q[j] : -__builtin_inff();
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = i < g.per_lane && e0 + i < E ? lt[e0 + i] : -__builtin_inff();
  }
  // what the choice needs: scores only where a bias or a sum meets them
  const bool by_score = g.bias != nullptr || (g.G > 1 && g.group_top == 2);
  bool odd = false;  // something fp32 cannot decide
#pragma unroll
  for (int i = 0; i < V; ++i) odd |= !(l[i] < __builtin_inff());  // NaN or +inf
  float top = 0.0f, sum = 1.0f, slack = 0.0f;
  float c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = l[i];
  if (g.score == 0 && (by_score || !g.renorm)) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
    top = row_max(m);
    odd |= top == -__builtin_inff();
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = __expf(l[i] - top);
      sum += c[i];
    }
    sum = row_add(sum);
  }
  if (by_score) {
    const float inv = __builtin_amdgcn_rcpf(sum);
    // |error| of a softmax score: (2.5 |d| + 40) 2^-24 s, d its logit's distance from the largest
    // (argument and result of exp, the sum of E terms, the quotient), at most 2.5 2^-20 of the
    // largest score 1 / sum; of a sigmoid 5 2^-24.  Twice that between two scores.
    slack = g.score == 0 ? inv * 0x1p-17f : 0x1p-20f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float sc = g.score == 0 ? c[i] * inv : __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));
      float b = 0.0f;
      if (g.bias != nullptr && i < g.per_lane && e0 + i < E) b = g.bias[e0 + i];
      odd |= !(fabsf(b) < __builtin_inff());
      c[i] = l[i] == -__builtin_inff() ? -__builtin_inff() : sc + b;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i];
  }
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    key[i] = i < g.per_lane && e0 + i < E ? (order_key32(c[i]) & ~15u) | (uint32_t)(15 - i) : 0u;
  sort_down(key);
  if (g.G > 1) {
    float a, b = -__builtin_inff();
    const int lpg = kRow / g.G;  // lanes per group, where groups are whole lanes
    if (g.on_lanes) {
      a = key_value(key[0]);
      if (V > 1) b = key_value(key[V > 1 ? 1 : 0]);
      for (int o = 1; o < lpg; o <<= 1) {
        const float a2 = __shfl_xor(a, o, kRow), b2 = __shfl_xor(b, o, kRow);
        b = fmaxf(fminf(a, a2), fmaxf(b, b2));
        a = fmaxf(a, a2);
      }
    } else {
      float* cs = (float*)s.value[wv][tok];
      const int size = E / g.G;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < g.per_lane && e0 + i < E) cs[e0 + i] = c[i];
      wave_lds_order();
      a = -__builtin_inff();
      if (li < g.G)
        for (int j = 0; j < size; ++j) {
          const float v = cs[li * size + j];
          b = fmaxf(b, fminf(a, v));
          a = fmaxf(a, v);
        }
    }
    const bool two = g.group_top == 2 && b > -__builtin_inff();
    const float worth = two ? a + b : a;
    const float size_of = a > -__builtin_inff() ? fabsf(a) + (two ? fabsf(b) : 0.0f) : 0.0f;
    const float near = 2.5f * 0x1p-19f * row_max(size_of) + 2.0f * slack;
    if (g.on_lanes ? li % lpg == 0 : li < g.G) s.group[wv][tok][g.on_lanes ? li / lpg : li] = worth;
    wave_lds_order();
    int above = 0, not_below = -1;  // groups surely above this lane's, and those not surely below but itself
    for (int j = 0; j < g.G; ++j) {
      const float o = s.group[wv][tok][j];
      above += o > worth + near ? 1 : 0;
      not_below += o < worth - near ? 0 : 1;
    }
    const bool has = g.on_lanes || li < g.G;
    bool keep = above < g.top_groups;
    odd |= has && keep != (not_below < g.top_groups);
    if (!g.on_lanes) {
      const uint32_t kept = (uint32_t)(__ballot(has && keep) >> (kRow * tok)) & 0xffffu;
      const int size = E / g.G;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int at = e0 + 15 - (int)(key[i] & 15u);
        if (key[i] != 0 && !((kept >> (at / size)) & 1)) key[i] = (kKeyNegInf & ~15u) | (key[i] & 15u);
      }
      sort_down(key);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] != 0 && !keep) key[i] = (kKeyNegInf & ~15u) | (key[i] & 15u);
    }
  }
  // the k + 1 best in turn; lane r keeps the r-th
  const int rounds = k < E ? k + 1 : k;
  uint32_t mine = 0, last = 0;
  for (int r = 0; r < rounds; ++r) {
    const uint32_t m = row_max(key[0]);
    const bool won = key[0] == m;
    odd |= __popcll(__ballot(won)) != 4;  // two lanes with one key: a tie
    if (won && r < k) s.sel[wv][tok][r] = e0 + 15 - (int)(m & 15u);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = won ? (i + 1 < V ? key[i + 1] : 0u) : key[i];
    if (li == r) mine = m;
    last = m;
  }
  {
    const float v = key_value(mine & ~15u);
    uint32_t after = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mine, 0x101, 0xf, 0xf, false);  // row_shl:1
    if (li == k - 1) after = last;
    const float n = key_value(after & ~15u);
    const float size_of = fmaxf(fabsf(v), n > -__builtin_inff() ? fabsf(n) : 0.0f);
    const bool pair = li < k - 1 || (li == k - 1 && k < E);
    odd |= pair && !(v - n > 1.25f * 0x1p-19f * size_of + slack + 1e-30f);
    odd |= li < k && !(v > -__builtin_inff());
  }
  if (__ballot(odd)) choose_exactly<V>(g, lt, wv, tok, li, s);
  wave_lds_order();
  const bool on = li < k;
  const int e = on ? s.sel[wv][tok][li] : 0;
  const float le = lt[e];
  bool poisoned = false;  // softmax: a NaN or +inf anywhere leaves no score
  if (g.score == 0) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) bad |= !(l[i] < __builtin_inff());
    poisoned = ((__ballot(bad) >> (kRow * tok)) & 0xffff) != 0;
  }
  float we;
  if (g.renorm) {
    we = renormalized(log_score(g.score, le), on, poisoned);
  } else if (g.score == 0) {
    we = poisoned ? __builtin_nanf("") : (le > -__builtin_inff() ? expf(le - top) / sum : 0.0f);
  } else {
    we = 1.0f / (1.0f + expf(-le));
  }
  if (live && on) {
    g.idx[t * k + li] = e;
    g.w[t * k + li] = g.scale * we;
  }
}

// One wave per token: lanes j < k hold the selected pairs' terms, then every
// lane writes its experts' entries once.
__global__ __launch_bounds__(256) void route_scored_bwd_kernel(int T, int E, int k, int score, int renorm, float scale,
                                                               const float* __restrict__ logits,
                                                               const int32_t* __restrict__ idx,
                                                               const float* __restrict__ dg,
                                                               float* __restrict__ dl) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;  // whole wave
  const float* lt = logits + (size_t)t * E;
  const bool dense = score == 0 && !renorm;
  float m = 0.0f, sum = 1.0f;
  float l[4];
  if (dense) {
    m = -__builtin_inff();
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane + 64 * i;
      l[i] = e < E ? lt[e] : -__builtin_inff();
      nan |= l[i] != l[i];
      m = fmaxf(m, l[i]);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
    if (__ballot(nan)) m = __builtin_nanf("");
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      l[i] = l[i] == -__builtin_inff() ? 0.0f : expf(l[i] - m);  // NaN where the row is
      sum += l[i];
    }
    sum = wave_sum(sum);
  }
  int e_l = -1;
  float g = 0.0f, a = -__builtin_inff();
  if (lane < k) {
    const int e = idx[(size_t)t * k + lane];
    if (e >= 0 && e < E) {
      e_l = e;
      g = dg[(size_t)t * k + lane];
      a = lt[e];
    }
  }
  float d;
  float sg = 0.0f;  // dense: sum_i s_i g_i
  const bool avail = e_l >= 0 && a != -__builtin_inff();
  const float s = score == 0 ? 0.0f : 1.0f / (1.0f + expf(-a));
  if (renorm) {
    const float p = renormalized(log_score(score, a), lane < 16 && e_l >= 0, false);
    float pg = avail ? p * g : 0.0f;
    pg = wave_sum(lane < 16 ? pg : 0.0f);
    d = scale * p * (g - pg) * (score == 0 ? 1.0f : 1.0f - s);
  } else if (dense) {
    const float se = avail ? expf(a - m) / sum : 0.0f;
    sg = wave_sum(avail ? se * g : 0.0f);
    d = scale * se * g;
  } else {
    d = scale * g * s * (1.0f - s);
  }
  if (!avail) d = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    float v = 0.0f;
    if (dense) v = sum == 0.0f ? 0.0f : -scale * (l[i] / sum) * sg;
    for (int j = 0; j < k; ++j) {
      const int ej = __builtin_amdgcn_readlane(e_l, j);
      const float dj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(d), j));
      if (ej == e) v += dj;
    }
    if (e < E) dl[(size_t)t * E + e] = v;
  }
}

}  // namespace

hipError_t launch_route_scored(int T, int E, int k, int score, int n_groups, int top_groups, int group_top,
                               bool renormalize, float scale, const float* logits, const float* bias, int32_t* idx,
                               float* w, hipStream_t stream) {
  RouteArgs g{T, E, k, score, n_groups, top_groups, group_top, (int)renormalize, scale, logits, bias, idx, w, 0, 0, 0};
  g.per_lane = (E + kRow - 1) / kRow;
  g.quads = g.per_lane % 4 == 0 && E % 4 == 0 && ((uintptr_t)logits & 15) == 0;
  g.on_lanes = E % kRow == 0 && kRow % n_groups == 0;
  const dim3 grid((unsigned)(((int64_t)T + 15) / 16)), block(256);
  if (g.per_lane <= 1) MOE_LAUNCH((route_scored_kernel<1>), grid, block, 0, stream, g);
  else if (g.per_lane <= 2) MOE_LAUNCH((route_scored_kernel<2>), grid, block, 0, stream, g);
  else if (g.per_lane <= 4) MOE_LAUNCH((route_scored_kernel<4>), grid, block, 0, stream, g);
  else if (g.per_lane <= 8) MOE_LAUNCH((route_scored_kernel<8>), grid, block, 0, stream, g);
  else MOE_LAUNCH((route_scored_kernel<16>), grid, block, 0, stream, g);
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(int T, int E, int k, int score, bool renormalize, float scale, const float* logits,
                                   const int32_t* idx, const float* dg, float* dlogits, hipStream_t stream) {
  MOE_LAUNCH(route_scored_bwd_kernel, dim3((T + 3) / 4), dim3(256), 0, stream, T, E, k, score, (int)renormalize,
             scale, logits, idx, dg, dlogits);
  return hipGetLastError();
}

}  // namespace moe
