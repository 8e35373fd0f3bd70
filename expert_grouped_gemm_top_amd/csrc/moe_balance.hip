// moe_balance.hip -- the routers' balance loss, its per-expert counts and its
// gradient.
//
//   p_te = softmax over the experts, or sigmoid(l_te) / sum_j sigmoid(l_tj)
//   c_se = listings of e in sequence s,  P_se = mean of p_te over its n_s tokens
//   loss = alpha E / (k N) sum_s sum_e c_se P_se,  N = sum_s n_s
//   dl_te = dloss alpha E / (k N n_s) p_te (c_se - sum_j p_tj c_sj) [(1 - sigmoid(l_te))]
//
// Sixteen lanes share a token; one pass over the logits each way.  Sums run in
// one fixed order: a workgroup's rows, then the runs of a sequence.
#include <algorithm>

#include "moe_common.h"
#include "moe_launch.h"
#include "moe_rows.h"

namespace moe {

namespace {

// Rows [begin, end) of sequence s, within the batch whatever the offsets say.
struct Rows {
  int begin, end;
};
__device__ __forceinline__ Rows rows_of(const int32_t* __restrict__ offsets, int s, int T) {
  if (offsets == nullptr) return {0, T};
  const int b = min(max(offsets[s], 0), T);
  return {b, min(max(offsets[s + 1], b), T)};
}

// alpha E / (k N)
__device__ __forceinline__ double loss_factor(const BalanceArgs& g) {
  const int S = g.offsets == nullptr ? 1 : g.n_seq;
  const int N = g.offsets == nullptr ? g.T : min(max(g.offsets[S], 0), g.T) - min(max(g.offsets[0], 0), g.T);
  return N > 0 ? (double)g.alpha * g.E / ((double)g.k * N) : 0.0;
}

// One token's logits over its 16 lanes: N runs of R experts a lane (four where rows
// are 16-byte aligned), every sixteenth run; -inf past the last.
template <int R_, int N_>
struct Token {
  static constexpr int R = R_, N = N_;
  static constexpr bool QUAD = R == 4;
  float v[N][R];
  static __device__ __forceinline__ int expert(int i, int li) { return R * (li + kRow * i); }
  __device__ __forceinline__ void load(const float* __restrict__ l, int E, int li) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = expert(i, li);
      if (QUAD) {
        const f32x4 q = e < E ? *(const f32x4*)(l + e) : f32x4{-1.f, -1.f, -1.f, -1.f} * __builtin_inff();
#pragma unroll
        for (int j = 0; j < R; ++j) v[i][j] = q[j];
      } else {
        v[i][0] = e < E ? l[e] : -__builtin_inff();
      }
    }
  }
  __device__ __forceinline__ float top() const {
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) m = fmaxf(m, v[i][j]);
    return row_max(m);
  }
  // The logits become the experts' shares.  Sigmoids are scaled by exp(-M), M = min(top, 0), so that they do not
  // all underflow: 1 / (exp(M - l) + exp(M)).  A token without an available expert has shares 0; NaN stays.
  __device__ __forceinline__ void to_shares(int score, float top) {
    float m = score == 0 ? top : fminf(top, 0.0f);
    if (m == -__builtin_inff()) m = 0.0f;
    const float em = score == 0 ? 0.0f : quick_exp(m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) {
        v[i][j] = score == 0 ? quick_exp(v[i][j] - m) : __builtin_amdgcn_rcpf(quick_exp(m - v[i][j]) + em);
        sum += v[i][j];
      }
    sum = row_add(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) v[i][j] *= inv;
  }
};

// Sum of v over a workgroup of NT threads, in one order; every thread gets it.
template <int NT>
__device__ __forceinline__ double group_sum(double v, double* s) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  __syncthreads();  // a sum before it has been read
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < NT / 64; ++i) v += s[i];
  return v;
}

// Runs of rows that a workgroup sums up: the batch in blocks of `each` rows, cut again where a sequence ends.  Along
// the rows either the block or the sequence moves on, so block + sequence numbers the runs: a workgroup each, and a
// place among the partial sums.  So long sequences are shared out whatever others there are (500000 rows, nearly all of
// them in one of 1000 sequences: 127 us, 9600 where the workgroups were divided by sequences).
struct BalanceParts {
  int each, runs;  // runs: as many as there may be
  float* p;        // [runs][E]
  int32_t* c;      // [runs][E]
  double* loss;    // a term of each workgroup of the second kernel
  uint32_t* done;  // how many of them have ended, set to 0 by the first kernel
};

constexpr int kRowThreads = 1024, kRowsAtOnce = kRowThreads / kRow;

// The sequence of run j: the last one whose first run is not behind j.  64 places are looked at at a time.
__device__ __forceinline__ int sequence_of(const BalanceArgs& g, int each, int j) {
  int lo = 0;
  for (int left = g.n_seq; left > 1;) {
    const int step = (left + 63) / 64, at = lane_id() * step;
    bool before = false;
    if (at < left) before = (int)((uint32_t)rows_of(g.offsets, lo + at, g.T).begin / (uint32_t)each) + lo + at <= j;
    const int found = (int)__popcll(__ballot(before));  // (unsigned: none less one would be 2^32 - 1)
    const int last = max(found - 1, 0) * step;          // none: a run in front of the first sequence's, without rows
    lo += last;
    left = min(step, left - last);
  }
  return lo;
}

// Workgroup j: run j.  ONE: it is the only workgroup, and writes the results itself.
template <typename Tok, bool ONE>
__global__ __launch_bounds__(kRowThreads) void balance_rows_kernel(BalanceArgs g, BalanceParts part,
                                                                   int32_t* __restrict__ counts,
                                                                   float* __restrict__ mean_p, float* __restrict__ loss) {
  constexpr int NT = kRowThreads;
  __shared__ float s_p[NT / 64][kMaxExperts];
  __shared__ int s_c[kMaxExperts];
  __shared__ double s_sum[NT / 64];
  const int tid = threadIdx.x, li = tid & 15, run = blockIdx.x;
  if (!ONE && run == 0 && tid == 0) *part.done = 0;
  const int s = ONE ? 0 : sequence_of(g, part.each, run);
  const Rows rows = rows_of(g.offsets, s, g.T);
  const int n = rows.end - rows.begin;
  int64_t begin = rows.begin, end = rows.end;
  if (!ONE) {
    const int64_t block = (int64_t)(run - s) * part.each;
    begin = max(begin, block);
    end = min(end, block + part.each);
  }
  if (!ONE && begin >= end) return;
  for (int e = tid; e < kMaxExperts; e += NT) s_c[e] = 0;
  __syncthreads();
  float acc[Tok::N][Tok::R] = {};
  for (int64_t t = begin + (tid >> 4); t < end; t += NT / kRow) {
    if (li < g.k) {
      const int e = g.idx[t * g.k + li];
      if (e >= 0 && e < g.E) atomicAdd(&s_c[e], 1);  // whole numbers: any order
    }
    Tok tok;
    tok.load(g.logits + t * g.E, g.E, li);
    tok.to_shares(g.score, tok.top());
#pragma unroll
    for (int i = 0; i < Tok::N; ++i)
#pragma unroll
      for (int j = 0; j < Tok::R; ++j) acc[i][j] += tok.v[i][j];
  }
#pragma unroll
  for (int i = 0; i < Tok::N; ++i)
#pragma unroll
    for (int j = 0; j < Tok::R; ++j) {
      float v = acc[i][j];
      v += __shfl_xor(v, 16, kWave);
      v += __shfl_xor(v, 32, kWave);
      if ((tid & 63) < kRow) s_p[tid >> 6][Tok::expert(i, li) + j] = v;
    }
  __syncthreads();
  double term = 0.0;
  if (tid < g.E) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v += s_p[w][tid];
    if (ONE) {
      const float mean = n > 0 ? v / (float)n : 0.0f;
      counts[tid] = s_c[tid];
      mean_p[tid] = mean;
      term = (double)s_c[tid] * mean;
    } else {
      const size_t at = (size_t)run * g.E + tid;
      part.p[at] = v;
      part.c[at] = s_c[tid];
    }
  }
  if (!ONE) return;
  term = group_sum<NT>(term, s_sum);
  if (tid == 0) *loss = (float)(loss_factor(g) * term);
}

// Workgroup (j, s) joins the parts of sequence s for 32 experts; the last one to end adds all terms in order.
constexpr int kJoinCols = 32;
__global__ __launch_bounds__(1024) void balance_join_kernel(BalanceArgs g, BalanceParts part, int32_t* __restrict__ counts,
                                                            float* __restrict__ mean_p, float* __restrict__ loss) {
  __shared__ double s_p[32][kJoinCols];
  __shared__ int s_c[32][kJoinCols];
  __shared__ double s_sum[16];
  __shared__ bool s_last;
  const int tid = threadIdx.x, q = tid / kJoinCols, e = blockIdx.x * kJoinCols + tid % kJoinCols, s = blockIdx.y;
  const Rows rows = rows_of(g.offsets, s, g.T);
  const int n = rows.end - rows.begin;
  double p = 0.0;
  int c = 0;
  if (e < g.E && n > 0) {
    const int b0 = (uint32_t)rows.begin / (uint32_t)part.each, b1 = (uint32_t)(rows.end - 1) / (uint32_t)part.each;
    const size_t first = (size_t)(b0 + s) * g.E + e;
#pragma unroll 8
    for (int i = q; i <= b1 - b0; i += 32) {
      p += (double)part.p[first + (size_t)i * g.E];
      c += part.c[first + (size_t)i * g.E];
    }
  }
  s_p[q][tid % kJoinCols] = p;
  s_c[q][tid % kJoinCols] = c;
  __syncthreads();
  double term = 0.0;
  if (tid < kJoinCols && e < g.E) {
    p = 0.0;
    c = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      p += s_p[i][tid];
      c += s_c[i][tid];
    }
    const float mean = n > 0 ? (float)(p / n) : 0.0f;
    counts[(size_t)s * g.E + e] = c;
    mean_p[(size_t)s * g.E + e] = mean;
    term = (double)c * mean;
  }
  term = group_sum<1024>(term, s_sum);
  const uint32_t groups = gridDim.x * gridDim.y;
  if (tid == 0) {
    __hip_atomic_store(part.loss + blockIdx.y * gridDim.x + blockIdx.x, term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s_last = __hip_atomic_fetch_add(part.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == groups - 1;
  }
  __syncthreads();
  if (!s_last) return;
  term = 0.0;
  for (uint32_t i = tid; i < groups; i += 1024)
    term += __hip_atomic_load(part.loss + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  term = group_sum<1024>(term, s_sum);
  if (tid == 0) *loss = (float)(loss_factor(g) * term);
}

// The gradient.  c_e - sum_j p_j c_j is formed from differences to the likeliest
// expert's count, d_j = c_j - c_top: of a confident token's top expert it is
// -sum_{j != top} p_j d_j, without the difference of two large numbers.
template <typename Tok>
__global__ __launch_bounds__(256) void balance_bwd_kernel(BalanceArgs g, const int32_t* __restrict__ counts,
                                                          const float* __restrict__ dloss, const float* dl_add,
                                                          float* dlogits) {
  const int li = threadIdx.x & 15, S = g.offsets == nullptr ? 1 : g.n_seq;
  const float factor = (float)(loss_factor(g) * (dloss != nullptr ? (double)*dloss : 1.0));
  int s = -1;
  Rows rows{0, 0};
  int c[Tok::N][Tok::R];
  float each = 0.0f;
  for (int64_t t = (int64_t)group_id() * 16 + (threadIdx.x >> 4); t < g.T; t += (int64_t)gridDim.x * gridDim.y * 16) {
    if (t < rows.begin || t >= rows.end) {  // another sequence, or none
      int lo = 0, hi = S;                   // the last one that begins at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (g.offsets[mid] <= t) lo = mid; else hi = mid;
      }
      rows = rows_of(g.offsets, lo, g.T);
      s = t >= rows.begin && t < rows.end ? lo : -1;
      if (s < 0) rows = {0, 0};
      each = s < 0 ? 0.0f : factor / (float)(rows.end - rows.begin);
#pragma unroll
      for (int i = 0; i < Tok::N; ++i)
#pragma unroll
        for (int j = 0; j < Tok::R; ++j) {
          const int e = Tok::expert(i, li) + j;
          c[i][j] = s >= 0 && e < g.E ? counts[(int64_t)s * g.E + e] : 0;
        }
    }
    float d[Tok::N][Tok::R] = {};
    if (s >= 0) {
      Tok tok;
      tok.load(g.logits + t * g.E, g.E, li);
      const float top = tok.top();
      uint32_t c_top = 0;
      float rest[Tok::N][Tok::R];  // 1 - sigmoid
#pragma unroll
      for (int i = 0; i < Tok::N; ++i)
#pragma unroll
        for (int j = 0; j < Tok::R; ++j) {
          if (tok.v[i][j] == top) c_top = max(c_top, (uint32_t)c[i][j]);
          rest[i][j] = g.score == 0 ? 1.0f : __builtin_amdgcn_rcpf(1.0f + quick_exp(tok.v[i][j]));
        }
      c_top = row_max(c_top);
      tok.to_shares(g.score, top);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < Tok::N; ++i)
#pragma unroll
        for (int j = 0; j < Tok::R; ++j) sum += tok.v[i][j] * (float)(c[i][j] - (int)c_top);
      sum = row_add(sum);
#pragma unroll
      for (int i = 0; i < Tok::N; ++i)
#pragma unroll
        for (int j = 0; j < Tok::R; ++j)
          d[i][j] = each * tok.v[i][j] * rest[i][j] * ((float)(c[i][j] - (int)c_top) - sum);
    } else if (dl_add == dlogits) {
      continue;  // nothing to add
    }
#pragma unroll
    for (int i = 0; i < Tok::N; ++i) {
      const int e = Tok::expert(i, li);
      if (e >= g.E) continue;
      const int64_t at = t * g.E + e;
      if (Tok::QUAD) {
        f32x4 v = {d[i][0], d[i][1 % Tok::R], d[i][2 % Tok::R], d[i][3 % Tok::R]};
        if (dl_add != nullptr) v += *(const f32x4*)(dl_add + at);
        *(f32x4*)(dlogits + at) = v;
      } else {
        dlogits[at] = d[i][0] + (dl_add != nullptr ? dl_add[at] : 0.0f);
      }
    }
  }
}

// Rows of a block: 512 of them share the batch out, each a multiple of what a workgroup takes at once (65536 rows of 128
// experts, both kernels: 15.3 us, 20.1 by 1024 blocks, 14.3 by 256; 131072 rows in 32 sequences 24.8, 22.9, 25.4; 65536 of
// 256 experts in 16 sequences 22.3, 25.6, 25.4), up to 8192, so that a thread adds at most 128 rows in fp32; the runs are
// added in 64 bits.
int balance_each(int T) {
  constexpr int64_t kBlocks = 512;
  return (int)std::min<int64_t>((T + kBlocks * kRowsAtOnce - 1) / (kBlocks * kRowsAtOnce) * kRowsAtOnce, 8192);
}
constexpr int kOneGroupRows = 256;  // up to here one workgroup does it all
int join_groups(int E) { return (E + kJoinCols - 1) / kJoinCols; }

bool balance_alone(int T, int n_seq) { return n_seq == 1 && T <= kOneGroupRows; }

BalanceParts balance_parts(int T, int E, int n_seq, void* ws, size_t* bytes) {
  char* at = (char*)ws;
  BalanceParts p;
  p.each = balance_each(T);
  p.runs = (int)(((int64_t)T + p.each - 1) / p.each) + n_seq - 1;
  const size_t n = (size_t)p.runs * E * 4;
  p.loss = (double*)at;
  at += (size_t)n_seq * join_groups(E) * sizeof(double);
  p.done = (uint32_t*)at;
  at += 16;
  p.p = (float*)at;
  at += n;
  p.c = (int32_t*)at;
  at += n;
  *bytes = ((size_t)(at - (char*)ws) + 15) / 16 * 16;
  return p;
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int n_seq) {
  if (balance_alone(T, n_seq)) return 0;
  size_t bytes;
  balance_parts(T, E, n_seq, nullptr, &bytes);
  return bytes;
}

// Runs f for the runs of experts that E and the rows' alignment ask for.
template <typename Fn>
static hipError_t with_token(int E, bool aligned, Fn&& f) {
  if (!aligned || E % 4 != 0) return f(Token<1, 16>{});
  if (E <= 64) return f(Token<4, 1>{});
  if (E <= 128) return f(Token<4, 2>{});
  return f(Token<4, 4>{});
}

hipError_t launch_balance_fwd(const BalanceArgs& g, int32_t* counts, float* mean_p, float* loss, void* ws,
                              hipStream_t stream) {
  const bool aligned = ((uintptr_t)g.logits & 15) == 0;
  if (balance_alone(g.T, g.n_seq))
    return with_token(g.E, aligned, [&](auto tok) {
      MOE_LAUNCH((balance_rows_kernel<decltype(tok), true>), dim3(1), dim3(kRowThreads), 0, stream, g, BalanceParts{},
                 counts, mean_p, loss);
      return hipGetLastError();
    });
  size_t bytes;
  const BalanceParts part = balance_parts(g.T, g.E, g.n_seq, ws, &bytes);
  hipError_t err = with_token(g.E, aligned, [&](auto tok) {
    MOE_LAUNCH((balance_rows_kernel<decltype(tok), false>), dim3(part.runs), dim3(kRowThreads), 0, stream, g, part, counts,
               mean_p, loss);
    return hipGetLastError();
  });
  if (err != hipSuccess) return err;
  MOE_LAUNCH(balance_join_kernel, dim3(join_groups(g.E), g.n_seq), dim3(1024), 0, stream, g, part, counts, mean_p, loss);
  return hipGetLastError();
}

hipError_t launch_balance_bwd(const BalanceArgs& g, const int32_t* counts, const float* dloss, const float* dl_add,
                              float* dlogits, hipStream_t stream) {
  const bool aligned = (((uintptr_t)g.logits | (uintptr_t)dl_add | (uintptr_t)dlogits) & 15) == 0;
  const dim3 grid((unsigned)std::min<int64_t>(((int64_t)g.T + 15) / 16, 1 << 14)), block(256);
  return with_token(g.E, aligned, [&](auto tok) {
    MOE_LAUNCH(balance_bwd_kernel<decltype(tok)>, grid, block, 0, stream, g, counts, dloss, dl_add, dlogits);
    return hipGetLastError();
  });
}

}  // namespace moe
