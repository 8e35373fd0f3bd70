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

// Key whose order as an unsigned number is the order of a 64-bit value: -0
// equals +0, every NaN is the largest key, -inf is above zero (no value).
__device__ __forceinline__ uint64_t order_key64(double v) {
  if (v != v) return ~0ull;
  const uint64_t u = (uint64_t)__double_as_longlong(v == 0.0 ? 0.0 : v);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmax(v, __shfl_xor(v, o, kWave));
  return v;
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// The log of a score up to a term that every expert of the token shares (none
// for sigmoid): differences of these are exact where the scores underflow.
__device__ __forceinline__ float log_score(int score, float l) {
  if (score == 0) return l;
  return fminf(l, 0.0f) - log1pf(expf(-fabsf(l)));
}

// Renormalised weight of each lane's selected score (lanes < k), the others 0:
// exp(a - max a) / sum, zeros where every selected score is zero.
__device__ __forceinline__ float renormalized(float a, bool on, bool poisoned) {
  float m = on ? a : -__builtin_inff();
  bool nan = poisoned || (on && a != a);
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 16));
  float e = (on && m > -__builtin_inff()) ? expf(a - m) : 0.0f;
  if (nan) e = __builtin_nanf("");
  float sum = e;
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 16);
  return sum == 0.0f ? 0.0f : e / sum;
}

// One wave per token, everything in 64 bits; lane l holds experts l + 64 i.
__global__ __launch_bounds__(256) void route_scored_kernel(int T, int E, int k, int score, int G, int top_groups,
                                                           int group_top, int renorm, float scale,
                                                           const float* __restrict__ logits,
                                                           const float* __restrict__ bias, int32_t* __restrict__ idx,
                                                           float* __restrict__ w) {
  __shared__ double s_c[4][kMaxExperts];
  __shared__ uint64_t s_key[4][kMaxExperts];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wv;
  if (t >= T) return;  // the whole wave; only this wave's LDS rows are used below
  const float* lt = logits + (size_t)t * E;
  float l[4];
  double s[4], c[4];
  double m = -__builtin_inf(), sum = 0.0;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < E ? lt[e] : -__builtin_inff();
    nan |= l[i] != l[i];
    m = fmax(m, (double)l[i]);
  }
  m = wave_max_f64(m);
  const bool poisoned = score == 0 && (__ballot(nan) != 0 || m == __builtin_inf());
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (score == 0) s[i] = l[i] > -__builtin_inff() ? exp((double)l[i] - m) : 0.0;
    else s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    sum += s[i];
  }
  if (score == 0) {
    sum = wave_sum_f64(sum);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = poisoned ? __builtin_nan("") : (sum > 0.0 ? s[i] / sum : 0.0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    if (e >= E) continue;
    c[i] = l[i] == -__builtin_inff() ? -__builtin_inf() : s[i] + (bias != nullptr ? (double)bias[e] : 0.0);
    s_c[wv][e] = c[i];
    // without a bias the logits' own order, which rounding of s cannot blur
    s_key[wv][e] = order_key64(bias != nullptr ? c[i] : (double)l[i]);
  }
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  if (G > 1) {
    const int size = E / G;
    uint64_t worth = 0;
    if (lane < G) {
      if (group_top == 1) {
        for (int j = 0; j < size; ++j) worth = max(worth, s_key[wv][lane * size + j]);
      } else {
        double a = -__builtin_inf(), b = -__builtin_inf();
        bool bad = false;
        for (int j = 0; j < size; ++j) {
          const double v = s_c[wv][lane * size + j];
          bad |= v != v;
          b = fmax(b, fmin(a, v));
          a = fmax(a, v);
        }
        worth = order_key64(bad ? __builtin_nan("") : (b > -__builtin_inf() ? a + b : a));
      }
    }
    int rank = 0;
    for (int g = 0; g < G; ++g) {
      const uint64_t o = __shfl(worth, g, kWave);
      rank += (o > worth || (o == worth && g < lane)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < G && rank < top_groups);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((kept >> (e / size)) & 1)) s_key[wv][e] = order_key64(-__builtin_inf());
    }
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  }
  uint64_t key[4];
  int rank[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) key[i] = lane + 64 * i < E ? s_key[wv][lane + 64 * i] : 0;
  for (int j = 0; j < E; ++j) {
    const uint64_t q = s_key[wv][j];
#pragma unroll
    for (int i = 0; i < 4; ++i) rank[i] += (q > key[i] || (q == key[i] && j < lane + 64 * i)) ? 1 : 0;
  }
  int32_t* s_sel = (int32_t*)s_c[wv];  // the choice scores are used up
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    if (e < E && rank[i] < k) s_sel[rank[i]] = e;
  }
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  const bool on = lane < k;
  const int e = on ? s_sel[lane] : 0;
  const float le = lt[e];
  float we;
  if (renorm) {
    we = renormalized(log_score(score, le), on, poisoned);
  } else if (score == 0) {
    we = poisoned ? __builtin_nanf("") : (sum > 0.0 && le > -__builtin_inff() ? (float)(exp((double)le - m) / sum) : 0.0f);
  } else {
    we = 1.0f / (1.0f + expf(-le));
  }
  if (on) {
    idx[(size_t)t * k + lane] = e;
    w[(size_t)t * k + lane] = scale * we;
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
  MOE_LAUNCH(route_scored_kernel, dim3((T + 3) / 4), dim3(256), 0, stream, T, E, k, score, n_groups, top_groups,
             group_top, (int)renormalize, scale, logits, bias, idx, w);
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(int T, int E, int k, int score, bool renormalize, float scale, const float* logits,
                                   const int32_t* idx, const float* dg, float* dlogits, hipStream_t stream) {
  MOE_LAUNCH(route_scored_bwd_kernel, dim3((T + 3) / 4), dim3(256), 0, stream, T, E, k, score, (int)renormalize,
             scale, logits, idx, dg, dlogits);
  return hipGetLastError();
}

}  // namespace moe
