// moe_vocab.hip -- softmax cross entropy over a vocabulary, without keeping the
// logits, and its gradients.
//
//   l_tv = x_t W_v,  loss_t = log sum_v exp(l_tv) - l_ty,  y = target[t]
//   dz_tv = f_t (q_tv - [v = y]),  dx = c dz W^T,  dW = c x^T dz
//
// Tokens that are not counted are left out of every product: the first kernel
// lists the others.  The forward's tiles of logits leave one maximum and sum of
// exponentials per row and run of columns.  The backward goes over the vocabulary
// in pieces: a piece's logits again, from them its dz, then both gradients' products
// with it.
//
// The target is kept apart from the other classes.  With rest = sum_{v != y} exp(l_v - l_y)
// the loss is log(1 + rest); the gradient is the others' softmax q (q_y = 0, sum 1)
// less the target's 1, times the others' probability f = rest / (1 + rest) =
// -expm1(-loss), and the token's weight.  All have their digits where a confident
// token's p is next to 1.
//
// The products take q - [v = y], rounded to the element type: its -1 is exact, and
// the others' roundings go in all directions.  f is multiplied to dx's sums, and for
// dW, which sums over the tokens, to their rows of x: rounded once more there
// (bf16: dW is 2.4e-3 of its norm off, dx 1.7e-3, of which 1.7e-3 by their own
// rounding).
//
// With few rows HBM bounds it: the forward of 128 over 2048 x 131072 reads W at 5.2
// TB/s (103 us), the frozen head's backward twice at 4.8 (226 us).  With many the
// matrix cores' feeding through LDS does: 1.1 PFLOP/s over the forward's 256 x 256
// tiles, 1.13 to 1.22 over the backward's three products of 8192 x 4096 x 65536 (10.8 to
// 11.7 ms, over boxes).
#include <algorithm>

#include "moe_common.h"
#include "moe_launch.h"
#include "moe_rows.h"
#include "moe_tile.h"
#include "moe_vocab_plan.h"

namespace moe {

namespace {

// The counted tokens, in order.
struct Listed {
  int32_t* head;  // [0] their number, [1] a ticket, set to 0
  int32_t* rows;  // [n] token
  int32_t* place; // [T] place of a token, -1 where not counted
  int32_t* y;     // [n] target
  float* off;     // [n] backward: log of the others' sum of exponentials
  float* f;       // [n] backward: their probability times the token's weight
};

// What they are listed from.
struct Tokens {
  int T, vocab;
  const int32_t* target;
  float *loss_out, *lse_out;         // forward: become 0 for tokens that are not counted
  const float *loss, *lse, *dloss;   // backward
  __device__ __forceinline__ int y(int64_t t) const {
    const int v = t < T ? target[t] : -1;
    return v >= 0 && v < vocab ? v : -1;
  }
  __device__ __forceinline__ float f(int64_t t) const {
    const float f = -expm1f(-loss[t]);
    return dloss != nullptr ? dloss[t] * f : f;
  }
  __device__ __forceinline__ float off(int64_t t) const {
    const float f = -expm1f(-loss[t]);
    return f == 0.0f ? __builtin_inff() : lse[t] + logf(f);  // a loss of 0: no gradient
  }
  __device__ __forceinline__ bool bwd() const { return loss != nullptr; }
};

// RUN neighbouring tokens a thread from `first` on: their targets and this thread's place among the listed.
// s_wave: an int a wave.
template <int NT, int RUN>
__device__ __forceinline__ int place_of(const Tokens& g, int64_t first, int (&y)[RUN], int& before, int* s_wave) {
  int mine = 0;
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    y[j] = g.y(first + j);
    mine += y[j] >= 0;
  }
  const int upto = wave_inclusive_scan(mine), w = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 63) s_wave[w] = upto;
  __syncthreads();
  int at = before + upto - mine;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) {
    at += i < w ? s_wave[i] : 0;
    before += s_wave[i];
  }
  return at;
}

// A token of that place, or -1 for none, into the list in memory.
__device__ __forceinline__ void list_token(const Tokens& g, const Listed& out, int64_t t, int y, int at) {
  if (t >= g.T) return;
  out.place[t] = y >= 0 ? at : -1;
  if (y < 0) {
    if (!g.bwd()) g.loss_out[t] = g.lse_out[t] = 0.0f;
    return;
  }
  out.rows[at] = (int)t;
  out.y[at] = y;
  if (g.bwd()) {
    out.off[at] = g.off(t);
    out.f[at] = g.f(t);
  }
}

// Lists many tokens, `each` a workgroup (a multiple of 1024), each of which counts the ones before its own for itself: a
// launch that waits for nothing (8192 tokens, 5.6 us; by one workgroup 30).  Past 256 workgroups each takes more tokens, or
// the counting would grow with the square (16 Mi tokens of 16 classes: the call 97 -> 28 ms).
__global__ __launch_bounds__(1024) void vocab_list_kernel(Tokens g, Listed out, int each) {
  __shared__ int s_wave[16];
  const int64_t first = (int64_t)blockIdx.x * each;
  int mine = 0;
  for (int64_t t = threadIdx.x; t < first; t += 1024 * 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) mine += t + 1024 * j < first && g.y(t + 1024 * j) >= 0;
  }
  mine = wave_inclusive_scan(mine);
  if ((threadIdx.x & 63) == 63) s_wave[threadIdx.x >> 6] = mine;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) before += s_wave[i];
  for (int64_t t = first + threadIdx.x; t < first + each; t += 1024) {
    int y[1];
    const int at = place_of<1024>(g, t, y, before, s_wave);
    list_token(g, out, t, y[0], at);
  }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) {
    out.head[0] = before;
    out.head[1] = 0;
  }
}

// Up to this many tokens every workgroup of the first product lists them for itself (in LDS), and one for the later
// kernels: a launch less (fp32 backward of 333 tokens 27 -> 21 us).
constexpr int kOwnListRows = 1024;
constexpr size_t kOwnListBytes = kOwnListRows * 12 + 64;
__device__ __forceinline__ int list_here(const Tokens& g, Listed& list, bool write, unsigned char* s) {
  int* s_wave = reinterpret_cast<int*>(s);
  int32_t* s_rows = reinterpret_cast<int32_t*>(s + 64);
  int32_t* s_y = s_rows + kOwnListRows;
  float* s_off = reinterpret_cast<float*>(s_y + kOwnListRows);
  constexpr int RUN = kOwnListRows / kTileThreads;
  int y[RUN], n = 0;
  const int64_t first = (int64_t)threadIdx.x * RUN;
  int at = place_of<kTileThreads>(g, first, y, n, s_wave);
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    if (write) list_token(g, list, first + j, y[j], at);
    if (y[j] < 0) continue;
    s_rows[at] = (int)(first + j);
    s_y[at] = y[j];
    if (g.bwd()) s_off[at] = g.off(first + j);
    ++at;
  }
  if (write && threadIdx.x == 0) {
    list.head[0] = n;
    list.head[1] = 0;
  }
  __syncthreads();
  list.rows = s_rows;
  list.y = s_y;
  list.off = s_off;
  return n;
}

template <typename T>
__device__ __forceinline__ float exp_of(float v) {
  return sizeof(T) == 4 ? expf(v) : quick_exp(v);
}

// ---- the forward ----------------------------------------------------------------

// A row's maximum over a run of columns, its target's left out, and the sum of exponentials above it.
struct Run {
  float top, sum;
};
// Two runs of columns as one.  A NaN is in a sum, where it stays.
__device__ __forceinline__ Run joined(const Run& a, const Run& b) {
  const float top = fmaxf(a.top, b.top), base = top == -__builtin_inff() ? 0.0f : top;
  return {top, a.sum * expf(a.top - base) + b.sum * expf(b.top - base)};
}

// Whether a workgroup takes tile after tile of logits, the next one's loads under what becomes of the last one's sums
// (128 rows of 2048 by 131072 columns: the loss 108 -> 104 us, the frozen head's backward 232 -> 226).  At 256 x 256 the
// addresses do not fit beside the sums, and spilled ones cost more (loss of 4096 rows: 1181 -> 1295 us).
template <typename T, typename C>
constexpr bool streams = sizeof(T) == 2 && C::KG == 1 && C::BM * C::BN < 256 * 256;

// Row statistics of a tile of logits.  Tiles of one reduction group (bf16) take them
// from the waves' registers; where the groups' sums must be joined first they
// come by eight columns.  At 256 x 256 over 2048 a tile's statistics cost
// 3 of its 58 us (through LDS 7).
// LDS behind the stage buffers: the waves' statistics [WN][BM], then the targets of the tile's rows [BM].
template <typename C>
constexpr int kTileRuns = C::BM * (C::NW / C::WM);

template <typename T>
struct LossOut {
  template <typename C>
  static constexpr bool kWhole = sizeof(T) == 2 && C::KG == 1;
  template <typename C>
  static constexpr size_t kBehind = kWhole<C> ? kTileRuns<C> * sizeof(Run) + C::BM * 4 : 0;
  int n, vocab, pitch;
  const int32_t* y;
  float* own;  // [n] the targets' logits
  Run* runs;   // [run][pitch rows]
  unsigned char* behind;

  template <typename C>
  __device__ __forceinline__ int32_t* targets() const {
    return reinterpret_cast<int32_t*>(behind + kTileRuns<C> * sizeof(Run));
  }
  template <typename C>
  __device__ __forceinline__ void ahead(int m0) const {
    const int m = m0 + (int)threadIdx.x;
    if (threadIdx.x < C::BM) targets<C>()[threadIdx.x] = m < n ? y[m] : -1;
  }
  template <typename C, int MI, int NJ>
  __device__ __forceinline__ void tile(f32x16 (&acc)[MI][NJ], int m0, int n0, unsigned char*) const {
    constexpr int BM = C::BM, WN = C::NW / C::WM, TM = BM / C::WM, TN = C::BN / WN;
    const int tid = threadIdx.x, l32 = tid & 31, hk = (tid >> 5) & 1, w = tid >> 6, wm = w % C::WM, wn = w / C::WM;
    const int first = n0 + TN * wn;  // this wave's columns
    Run* s_run = reinterpret_cast<Run*>(behind);  // [WN][BM]
    const int32_t* target = targets<C>();
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int row = TM * wm + 32 * i + l32, m = m0 + row;
      const int at = target[row] - first;  // the target, if it is among them
      if (__ballot(at >= 0 && at < TN) || first + TN > vocab) {  // a few waves, or the last columns
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int col = 32 * j + 8 * (r / 4) + 4 * hk + r % 4;
            if (at == col) own[m] = acc[i][j][r];
            if (at == col || first + col >= vocab) acc[i][j][r] = -__builtin_inff();
          }
      }
      float top = -__builtin_inff();
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, acc[i][j][r]);
      top = fmaxf(top, __shfl_xor(top, 32, kWave));
      const float base = top == -__builtin_inff() ? 0.0f : top * 1.44269504f;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) sum += __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], 1.44269504f, -base));
      sum += __shfl_xor(sum, 32, kWave);
      if (hk == 0) s_run[wn * BM + row] = Run{top, sum};
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the waves' statistics are written
    barrier_no_fence();
    if (tid < BM && m0 + tid < n) {
      Run a = s_run[tid];
#pragma unroll
      for (int i = 1; i < WN; ++i) a = joined(a, s_run[i * BM + tid]);
      runs[(int64_t)(n0 / C::BN) * pitch + m0 + tid] = a;
    }
  }

  __device__ __forceinline__ bool skip(int, int) const { return false; }
  template <typename Lanes>
  __device__ __forceinline__ void operator()(int64_t m, int n0, float (&v)[8], Lanes) const {
    const int at = (m < n ? y[m] : -1) - n0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (at == j) own[m] = v[j];
      if (at == j || n0 + j >= vocab) v[j] = -__builtin_inff();
    }
    float top = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
#pragma unroll
    for (int o = Lanes::value / 2; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, kWave));
    const float base = top == -__builtin_inff() ? 0.0f : top;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += exp_of<T>(v[j] - base);
#pragma unroll
    for (int o = Lanes::value / 2; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, kWave);
    constexpr int COLS = 8 * Lanes::value;
    if (n0 % COLS == 0 && m < n && n0 < vocab) runs[(int64_t)(n0 / COLS) * pitch + m] = Run{top, sum};
  }
};

template <typename T>
struct LogitsArgs {
  TileSource g;  // M: the batch's tokens; b from the piece's first column on
  int K;
  Listed list;
  Tokens tokens;
  bool own_list;
};

// Tile of the counted tokens' rows; false past the last.
template <typename C>
__device__ __forceinline__ bool row_tile(int item, int n, int N, int& mt, int& nt) {
  const int mtiles = (n + C::BM - 1) / C::BM, ntiles = (N + C::BN - 1) / C::BN;
  if (item >= mtiles * ntiles) return false;
  tile_of(item, mtiles, ntiles, 1024 / C::BM, mt, nt);
  return true;
}

template <typename T, typename C, bool TAIL>
__global__ __launch_bounds__(kTileThreads, 2) void vocab_loss_kernel(LogitsArgs<T> a, int vocab, int pitch, float* own,
                                                                     Run* runs) {
  extern __shared__ __attribute__((aligned(16))) unsigned char s_dyn[];
  int item = group_id();
  TileSource g = a.g;
  Listed list = a.list;
  using Out = LossOut<T>;
  unsigned char* behind = s_dyn + C::LDS;
  g.M = a.own_list ? list_here(a.tokens, list, item == 0, behind + Out::template kBehind<C>) : list.head[0];
  g.rows = list.rows;
  const Out out{g.M, vocab, pitch, list.y, own, runs, behind};
  if constexpr (streams<T, C>) {
    auto next = [&](int& mt, int& nt) {
      const bool more = row_tile<C>(item, g.M, g.N, mt, nt);
      item += gridDim.x * gridDim.y;
      return more;
    };
    tile_products<T, true, false, C, TAIL, true>(g, next, 0, a.K, s_dyn, out);
  } else {
    int mt, nt;
    if (!row_tile<C>(item, g.M, g.N, mt, nt)) return;
    if constexpr (Out::template kWhole<C>) out.template ahead<C>(mt * C::BM);
    tile_product<T, true, false, C, TAIL>(g, mt, nt, 0, a.K, s_dyn, out);
  }
}

// Joins the runs of 16 rows per workgroup, 64 threads each; the last workgroup adds up the mean.
struct JoinArgs {
  int n_runs, pitch;
  const Run* runs;
  const float* own;
  Listed list;
  double* part;  // a sum of losses of each workgroup
  float *loss, *lse, *mean;
};
__global__ __launch_bounds__(1024) void vocab_join_kernel(JoinArgs a) {
  __shared__ Run s_run[64][17];
  __shared__ double s_loss[16];
  __shared__ bool s_last;
  const int tid = threadIdx.x, r = tid & 15, q = tid >> 4, n = a.list.head[0];
  const int row = blockIdx.x * 16 + r;
  const int groups = max(1, (n + 15) / 16);
  if ((int)blockIdx.x >= groups) return;
  Run run{-__builtin_inff(), 0.0f};
  for (int first = q; first < a.n_runs; first += 64 * 8) {  // eight runs at a time
    Run some[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = first + 64 * k;
      some[k] = row < n && i < a.n_runs ? a.runs[(int64_t)i * a.pitch + row] : Run{-__builtin_inff(), 0.0f};
    }
    float top = run.top;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, some[k].top);
    const float base = top == -__builtin_inff() ? 0.0f : top;
    run = Run{top, run.sum * expf(run.top - base)};
#pragma unroll
    for (int k = 0; k < 8; ++k) run.sum += some[k].sum * expf(some[k].top - base);
  }
  s_run[q][r] = run;
  __syncthreads();
  // wave w joins row w: 64 runs over its lanes
  const int w = tid >> 6, lane = tid & 63;
  run = s_run[lane][w];
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) run = joined(run, Run{__shfl_xor(run.top, o, kWave), __shfl_xor(run.sum, o, kWave)});
  if (lane == 0) {
    const int at = blockIdx.x * 16 + w;
    float loss = 0.0f;
    if (at < n) {
      const float own = a.own[at], others = run.top + logf(run.sum), d = others - own;
      const float less = log1pf(expf(-fabsf(d)));
      loss = fmaxf(d, 0.0f) + less;
      const int t = a.list.rows[at];
      a.loss[t] = loss;
      a.lse[t] = fmaxf(others, own) + less;  // not own + loss: a target far below would take the others' digits
    }
    s_loss[w] = (double)loss;
  }
  __syncthreads();
  if (tid == 0) {
    double l = 0.0;
    for (int i = 0; i < 16; ++i) l += s_loss[i];
    __hip_atomic_store(a.part + blockIdx.x, l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s_last = __hip_atomic_fetch_add(a.list.head + 1, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == groups - 1;
  }
  __syncthreads();
  if (!s_last || tid >= 64) return;
  double l = 0.0;
  for (int i = tid; i < groups; i += 64) l += __hip_atomic_load(a.part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) l += __shfl_xor(l, o, kWave);
  if (tid == 0) {
    a.mean[0] = n > 0 ? (float)(l / n) : 0.0f;
    a.mean[1] = n > 0 ? (float)(1.0 / n) : 0.0f;
  }
}

// ---- the backward ---------------------------------------------------------------

// q - [v = y] of a tile of logits.
template <typename T>
struct GradOut {
  template <typename C>
  static constexpr bool kWhole = sizeof(T) == 2 && C::KG == 1;
  int n, first, vocab;  // the piece's first column
  int pitch;
  Listed list;
  T* dz;
  float2* rows;  // LDS, [BM] of the tile's rows, where it streams: log of the others' sum in base 2, target (its bits)

  __device__ __forceinline__ float2 row_of(int m) const {
    return m < n ? float2{list.off[m] * 1.44269504f, __int_as_float(list.y[m] - first)} : float2{0.0f, __int_as_float(-1)};
  }
  template <typename C>
  __device__ __forceinline__ void ahead(int m0) const {
    if (threadIdx.x < C::BM) rows[threadIdx.x] = row_of(m0 + (int)threadIdx.x);
  }
  template <typename C, int MI, int NJ>
  __device__ __forceinline__ void tile(f32x16 (&acc)[MI][NJ], int m0, int n0, unsigned char* s_dyn) const {
    constexpr int WN = C::NW / C::WM, TM = C::BM / C::WM, TN = C::BN / WN;
    const int wv = threadIdx.x >> 6;
    float base[MI];
    int at[MI];
    bool special = first + n0 + C::BN > vocab;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int row = TM * (wv % C::WM) + 32 * i + (threadIdx.x & 31);
      const float2 r = streams<T, C> ? rows[row] : row_of(m0 + row);
      base[i] = r.x;
      at[i] = __float_as_int(r.y) - n0;
      const int in_wave = at[i] - TN * (wv / C::WM);
      special |= __ballot(in_wave >= 0 && in_wave < TN) != 0;
    }
    if constexpr (streams<T, C>) {
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave has its rows
      barrier_no_fence();                   // ... and every wave: the next tile's may come
    }
    auto go = [&](auto with) {
      auto make = [&](int i, int, int col, float (&v)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = __builtin_amdgcn_exp2f(fmaf(v[e], 1.44269504f, -base[i]));
          if (decltype(with)::value) {
            if (first + n0 + col + e >= vocab) v[e] = 0.0f;
            if (at[i] == col + e) v[e] = -1.0f;
          }
        }
      };
      auto put = [&](int row, int col, u32x4 q) {
        if (m0 + row < n) *(u32x4*)(dz + (int64_t)(m0 + row) * pitch + n0 + col) = q;
      };
      if constexpr (streams<T, C>) leave_bf16_direct<C>(acc, make, put);
      else leave_bf16<C>(acc, s_dyn, make, put);
    };
    if (special) go(std::true_type{});  // a few waves, or the last columns
    else go(std::false_type{});
  }

  __device__ __forceinline__ bool skip(int m, int) const { return m >= n; }
  template <typename Lanes>
  __device__ __forceinline__ void operator()(int64_t m, int n0, float (&v)[8], Lanes) const {
    const float off = list.off[m];
    const int at = list.y[m] - first - n0, end = vocab - first - n0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = j < end ? exp_of<T>(v[j] - off) : 0.0f;
      if (j == at) v[j] = -1.0f;
    }
    store8(dz + m * pitch + n0, v);
  }
};

// What the first piece's launch does beside it, in workgroups of its own or behind their tiles: the listed tokens' rows of x times their f, one
// behind the other, for dW, which sums over them (out NULL: not wanted), and zeros for the other tokens' dx (NULL alike).
template <typename T>
struct Layout {
  int H;
  const T* x;
  T* out;
  T* dx;
  int64_t tiles;  // workgroups in front of these
  int groups;
};
template <typename T>
__device__ __forceinline__ void lay_out(const Layout<T>& g, const Tokens& tokens, const int32_t* rows, int n, int group) {
  const int lane = threadIdx.x & 63, step = g.groups * (kTileThreads / 64);
  const int first = group * (kTileThreads / 64) + (threadIdx.x >> 6);  // a wave per row
  if (g.out != nullptr)
    for (int r = first; r < n; r += step) {
      const int64_t t = rows[r];
      const float f = tokens.f(t);
      for (int i = 8 * lane; i < g.H; i += 8 * 64) {
        float v[8];
        load8(g.x + t * g.H + i, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= f;
        store8(g.out + (int64_t)r * g.H + i, v);
      }
    }
  if (g.dx != nullptr)
    for (int64_t t = first; t < tokens.T; t += step) {
      if (tokens.y(t) >= 0) continue;
      const float zero[8] = {};
      for (int i = 8 * lane; i < g.H; i += 8 * 64) store8(g.dx + t * g.H + i, zero);
    }
}

template <typename T, typename C, bool TAIL>
__global__ __launch_bounds__(kTileThreads, 2) void vocab_dz_kernel(LogitsArgs<T> a, int first, int pitch, T* dz,
                                                                   Layout<T> beside) {
  extern __shared__ __attribute__((aligned(16))) unsigned char s_dyn[];
  const int64_t item = group_id();
  TileSource g = a.g;
  Listed list = a.list;
  g.M = a.own_list ? list_here(a.tokens, list, item == 0, s_dyn + C::LDS) : list.head[0];
  g.rows = list.rows;
  GradOut<T> out{g.M, first, a.tokens.vocab, pitch, list, dz, nullptr};
  if constexpr (streams<T, C>) {
    out.rows = reinterpret_cast<float2*>(s_dyn + C::LDS + kOwnListBytes);
    int tile = (int)item;
    auto next = [&](int& mt, int& nt) {
      const bool more = row_tile<C>(tile, g.M, g.N, mt, nt);
      tile += (int)beside.tiles;
      return more;
    };
    if (item < beside.tiles) tile_products<T, true, false, C, TAIL, true>(g, next, 0, a.K, s_dyn, out);
    if (item < beside.groups) lay_out(beside, a.tokens, list.rows, g.M, (int)item);
  } else {
    if (item >= beside.tiles) {
      if (item - beside.tiles < beside.groups) lay_out(beside, a.tokens, list.rows, g.M, (int)(item - beside.tiles));
      return;
    }
    int mt, nt;
    if (!row_tile<C>((int)item, g.M, g.N, mt, nt)) return;
    tile_product<T, true, false, C, TAIL>(g, mt, nt, 0, a.K, s_dyn, out);
  }
}

// The factor that dz was held without.
struct Factor {
  float scale;
  const float* per_mean;  // {mean, 1 / n}; NULL where tokens are weighted one by one
  __device__ __forceinline__ float get() const { return per_mean != nullptr ? scale * per_mean[1] : scale; }
};

// Sums of dx over the pieces, [slice][pitch rows][H]; the last piece of a product in one slice leaves dx itself.
template <typename T>
struct DxOut {
  template <typename C>
  static constexpr bool kWhole = false;
  int n, H, pitch, slice;
  bool add;
  float* sums;
  const Listed& list;
  float c;
  T* dx;  // NULL: sums
  __device__ __forceinline__ bool skip(int m, int h) const { return m >= n || h >= H; }
  template <typename Lanes>
  __device__ __forceinline__ void operator()(int64_t m, int h, float (&v)[8], Lanes) const {
    float* at = sums + ((int64_t)slice * pitch + m) * H + h;
    if (add) {
      float u[8];
      load8(at, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += u[j];
    }
    if (dx == nullptr) return store8(at, v);
    const float f = c * list.f[m];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= f;
    store8(dx + (int64_t)list.rows[m] * H + h, v);
  }
};

template <typename T>
struct DwOut {
  template <typename C>
  static constexpr bool kWhole = sizeof(T) == 2 && C::KG == 1;
  int H, N;
  int64_t ld;
  float c;
  T* dw;
  template <typename C, int MI, int NJ>
  __device__ __forceinline__ void tile(f32x16 (&acc)[MI][NJ], int m0, int n0, unsigned char* s_dyn) const {
    leave_bf16<C>(
        acc, s_dyn,
        [&](int, int, int, float (&v)[4]) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] *= c;
        },
        [&](int row, int col, u32x4 q) {  // N is a multiple of 8: a run is all in or all out
          if (m0 + row < H && n0 + col < N) *(u32x4*)(dw + (int64_t)(m0 + row) * ld + n0 + col) = q;
        });
  }
  __device__ __forceinline__ bool skip(int h, int n) const { return h >= H || n >= N; }
  template <typename Lanes>
  __device__ __forceinline__ void operator()(int64_t h, int n, float (&v)[8], Lanes) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= c;
    store8(dw + h * ld + n, v);
  }
};

// The slices of dx's product.  They are laid out for the batch's tokens; where fewer are counted their tiles leave
// workgroups over, and each slice is cut into as many as those do, on the device, which knows the count (T 1703 with 307
// counted, H 360, V 42516, fp32: 1068 -> 538 us).  Their sums lie in the rows that are not needed either.
struct Slices {
  int many, slice;  // for the batch's tokens: how many, and their columns
  int tiles;        // ... and row tiles
  int piece;        // columns of all but the last piece
  int pitch;
  bool again;       // whether to cut them
  struct Cut {
    int slice, pitch, many;
  };
  __device__ __forceinline__ Cut cut(int n, int bm) const {
    const int times = again ? tiles / max(1, (n + bm - 1) / bm) : 1;
    if (times <= 1) return {slice, pitch, many};
    const int cols = (slice + times - 1) / times, c = (cols + 127) / 128 * 128;
    return {c, (n + bm - 1) / bm * bm, (piece + c - 1) / c};
  }
};

struct GradArgs {
  TileSource gx, gw;    // dz W^T (M: the batch's tokens) and x^T dz
  int Kx;               // the piece's columns
  Slices slices;
  Listed list;
  int add;              // not the first piece
  float* sums;
  void* dx;             // the last piece: written from here where there is one slice
  Factor c;
  void* dw;
  int64_t ldw;
  int64_t nx, nw;       // workgroups of each product
  int x_first;
};

// Both gradients' products with one piece of dz, in one launch as in linear_bwd_kernel.  dW sums over as many
// tokens as are counted: its last stage is masked.
template <typename T, typename CX, typename CW, bool TAIL>
__global__ __launch_bounds__(kTileThreads, 2) void vocab_grads_kernel(GradArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char s_dyn[];
  const int64_t b = group_id();
  const int n = a.list.head[0];
  const bool is_x = a.x_first ? b < a.nx : b >= a.nw;
  if (is_x) {
    TileSource g = a.gx;
    g.M = n;
    const int mtiles = (n + CX::BM - 1) / CX::BM, ntiles = (g.N + CX::BN - 1) / CX::BN, tiles = mtiles * ntiles;
    const int item = (int)(a.x_first ? b : b - a.nw);
    if (tiles == 0) return;
    const Slices::Cut cut = a.slices.cut(n, CX::BM);
    const int s = item / tiles;
    if (s * (int64_t)cut.slice >= a.Kx) return;
    const int kb = s * cut.slice;
    int mt, nt;
    tile_of(item % tiles, mtiles, ntiles, 1024 / CX::BM, mt, nt);
    tile_product<T, true, true, CX, TAIL>(g, mt, nt, kb, min(a.Kx, kb + cut.slice), s_dyn,
                                           DxOut<T>{n, g.N, cut.pitch, s, a.add != 0, a.sums, a.list, a.c.get(),
                                                    cut.many == 1 ? (T*)a.dx : nullptr});
  } else {
    const TileSource& g = a.gw;
    const int mtiles = (g.M + CW::BM - 1) / CW::BM, ntiles = (g.N + CW::BN - 1) / CW::BN;
    const int item = (int)(a.x_first ? b - a.nx : b);
    if (item >= mtiles * ntiles) return;
    int mt, nt;
    tile_of(item, mtiles, ntiles, 1024 / CW::BM, mt, nt);
    tile_product<T, false, false, CW, true>(g, mt, nt, 0, n, s_dyn, DwOut<T>{g.M, g.N, a.ldw, a.c.get(), (T*)a.dw});
  }
}

// dx of the counted tokens from the slices' sums.
template <typename T>
__global__ __launch_bounds__(256) void vocab_dx_kernel(int T_, int H, Slices slices, int bm, Listed list,
                                                       const float* __restrict__ sums, Factor f, T* __restrict__ dx) {
  const Slices::Cut cut = slices.cut(list.head[0], bm);
  if (cut.many == 1) return;  // the last piece has left dx
  const float c = f.get();
  const int runs = H / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)T_ * runs; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / runs;
    const int h = 8 * (int)(i % runs), place = list.place[t];
    if (place < 0) continue;
    float v[8] = {};
#pragma unroll 4
    for (int s = 0; s < cut.many; ++s) {
      float u[8];
      load8(sums + ((int64_t)s * cut.pitch + place) * H + h, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += u[j];
    }
    const float f = c * list.f[place];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= f;
    store8(dx + t * H + h, v);
  }
}

// ---- plans and launchers -----------------------------------------------------------

// kTile128x256, and dx's tile for few rows.
using FlatTile = Tile<128, 256, 8, 2, 1, 3>;
using DeepTile = Tile<128, 128, 8, 2, 1, 4>;

template <typename T, typename Fn>
hipError_t with_tile(int tile, Fn&& run) {
  if constexpr (sizeof(T) == 2) {
    if (tile == kTile128x256) return run(FlatTile{});
    if (tile == kTile256x256) return run(Tile0{});
    if (tile == kTile256x128) return run(Tile1{});
  }
  if (tile == kTile128x128) return run(Tile2{});
  if (tile == kTile128x64) return run(Tile3{});
  if (tile == kTile64x64) return run(Tile4<T>{});
  return run(Tile5{});
}

const VocabPlan& vocab_plan(int T, int H, int V, int esize, bool dx, bool dw) {
  return remembered<VocabPlan>(T, H, V, esize + (dx ? 8 : 0) + (dw ? 16 : 0),
                               [&] { return make_vocab_plan(T, H, V, esize, dx, dw); });
}

// The columns of a run that a tile of the forward leaves.
template <typename T>
int run_cols(int tile) {
  int cols = 0;
  (void)with_tile<T>(tile, [&](auto t) {
    using C = decltype(t);
    cols = LossOut<T>::template kWhole<C> ? C::BN : C::OUT_COLS;
    return hipSuccess;
  });
  return cols;
}

struct Space {
  Listed list;
  double* part;
  float* own;
  Run* runs;
  void *x, *dz;
  float* sums;
  size_t bytes;
};

// A workspace's parts: the list, then the forward's runs or the backward's piece.
Space vocab_space(void* ws, int T, int H, int V, int esize, const VocabPlan& p, bool bwd) {
  Space s{};
  char* at = (char*)ws;
  auto take = [&](size_t bytes) {
    char* here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t row = (size_t)T * 4;
  s.list.head = (int32_t*)take(256);
  s.list.rows = (int32_t*)take(row);
  s.list.place = (int32_t*)take(row);
  s.list.y = (int32_t*)take(row);
  if (!bwd) {
    s.part = (double*)take(((size_t)T + 15) / 16 * 8);
    s.own = (float*)take(row);
    const int cols = esize == 4 ? run_cols<float>(p.logits) : run_cols<uint16_t>(p.logits);
    s.runs = (Run*)take((size_t)((V + cols - 1) / cols) * p.pitch * sizeof(Run));
  } else {
    s.list.off = (float*)take(row);
    s.list.f = (float*)take(row);
    s.x = take((size_t)p.pitch * H * esize);
    s.dz = take((size_t)p.pitch * p.piece * esize);
    s.sums = (float*)take((size_t)std::max(1, p.grads.x.slices) * p.pitch * H * 4);
  }
  s.bytes = (size_t)(at - (char*)ws);
  return s;
}

template <typename Kern, typename... Args>
hipError_t run_tiles(Kern kern, size_t lds, int64_t groups, hipStream_t stream, PerDeviceOnce& once, Args... args) {
  hipError_t err = allow_dynamic_lds(once, (const void*)kern, lds);
  if (err != hipSuccess) return err;
  MOE_LAUNCH(kern, wide_grid(groups), dim3(kTileThreads), lds, stream, args...);
  return hipGetLastError();
}

template <typename C>
int64_t tiles_of(int M, int N) {
  return (int64_t)((M + C::BM - 1) / C::BM) * ((N + C::BN - 1) / C::BN);
}

hipError_t list_tokens(const Tokens& tokens, const Listed& list, hipStream_t stream) {
  const int each = rounded_up(((int64_t)tokens.T + kCus - 1) / kCus, 1024);
  MOE_LAUNCH(vocab_list_kernel, dim3((unsigned)((tokens.T + each - 1) / each)), dim3(1024), 0, stream, tokens, list, each);
  return hipGetLastError();
}

template <typename T, typename C, bool TAIL>
hipError_t run_loss(const LogitsArgs<T>& a, int vocab, int pitch, float* own, Run* runs, hipStream_t stream) {
  static PerDeviceOnce once;
  // the forward's list needs no `off`: the 128 x 256 tile leaves no more room
  constexpr size_t lds = C::LDS + LossOut<T>::template kBehind<C> + kOwnListBytes - 4 * kOwnListRows;
  static_assert(lds <= 160 * 1024, "one CU's LDS");
  int64_t groups = tiles_of<C>(a.g.M, a.g.N);
  if (streams<T, C>) groups = std::min<int64_t>(groups, kCus);  // each takes tile after tile
  return run_tiles(vocab_loss_kernel<T, C, TAIL>, lds, groups, stream, once, a, vocab, pitch, own, runs);
}

template <typename T, typename C, bool TAIL>
hipError_t run_dz(const LogitsArgs<T>& a, int first, int pitch, T* dz, Layout<T> beside, hipStream_t stream) {
  static PerDeviceOnce once;
  beside.tiles = tiles_of<C>(a.g.M, a.g.N);
  size_t lds = C::LDS + kOwnListBytes;
  int64_t groups = beside.tiles + beside.groups;
  if constexpr (streams<T, C>) {
    static_assert(C::LDS + kOwnListBytes + C::BM * sizeof(float2) <= 160 * 1024, "one CU's LDS");
    lds += C::BM * sizeof(float2);
    beside.tiles = std::min<int64_t>(beside.tiles, kCus);  // each takes tile after tile, then lays out its share
    groups = std::max<int64_t>(beside.tiles, beside.groups);
  }
  return run_tiles(vocab_dz_kernel<T, C, TAIL>, lds, groups, stream, once, a, first, pitch, dz, beside);
}

template <typename T, typename CX, typename CW, bool TAIL>
hipError_t run_grads(const GradArgs& a, hipStream_t stream) {
  static PerDeviceOnce once;
  return run_tiles(vocab_grads_kernel<T, CX, CW, TAIL>, std::max(CX::LDS, CW::LDS), a.nx + a.nw, stream, once, a);
}

template <typename T>
hipError_t vocab_fwd_typed(const VocabArgs& g, float* loss, float* lse, float* mean, void* ws, hipStream_t stream) {
  const VocabPlan& p = vocab_plan(g.T, g.H, g.V, sizeof(T), false, false);
  const Space s = vocab_space(ws, g.T, g.H, g.V, sizeof(T), p, false);
  const Tokens tokens{g.T, g.vocab, g.target, loss, lse, nullptr, nullptr, nullptr};
  const bool own_list = g.T <= kOwnListRows;
  hipError_t err = own_list ? hipSuccess : list_tokens(tokens, s.list, stream);
  if (err != hipSuccess) return err;
  // columns past the vocabulary's end need no product
  const int cols = std::min(g.V, rounded_up(g.vocab, 8));
  const LogitsArgs<T> a{{g.T, cols, g.x, g.H, g.w, g.V, s.list.rows}, g.H, s.list, tokens, own_list};
  err = with_tile<T>(p.logits, [&](auto tile) {
    using C = decltype(tile);
    const bool tail = g.H % (kStageK<T> * C::KG) != 0;
    return tail ? run_loss<T, C, true>(a, g.vocab, p.pitch, s.own, s.runs, stream)
                : run_loss<T, C, false>(a, g.vocab, p.pitch, s.own, s.runs, stream);
  });
  if (err != hipSuccess) return err;
  const int run = run_cols<T>(p.logits);
  const JoinArgs j{(cols + run - 1) / run, p.pitch, s.runs, s.own, s.list, s.part, loss, lse, mean};
  MOE_LAUNCH(vocab_join_kernel, dim3((g.T + 15) / 16), dim3(1024), 0, stream, j);
  return hipGetLastError();
}

template <typename T>
hipError_t vocab_bwd_typed(const VocabArgs& g, const float* loss, const float* lse, const float* mean, const float* dloss,
                           float scale, void* dx, void* dw, void* ws, hipStream_t stream) {
  const VocabPlan& p = vocab_plan(g.T, g.H, g.V, sizeof(T), dx != nullptr, dw != nullptr);
  const Space s = vocab_space(ws, g.T, g.H, g.V, sizeof(T), p, true);
  const Tokens tokens{g.T, g.vocab, g.target, nullptr, nullptr, loss, lse, dloss};
  const bool own_list = g.T <= kOwnListRows;
  hipError_t err = own_list ? hipSuccess : list_tokens(tokens, s.list, stream);
  if (err != hipSuccess) return err;
  const Factor c{scale, dloss != nullptr ? nullptr : mean};
  T* dz = (T*)s.dz;
  Slices slices{};
  int bm = 1;
  if (dx != nullptr) {
    slices.slice = p.grads.x.slice;
    slices.piece = std::min(p.piece, g.V);
    slices.many = (slices.piece + slices.slice - 1) / slices.slice;
    slices.pitch = p.pitch;
    slices.again = slices.many > 1 || !own_list;  // few tokens in one slice: not worth a launch
  }
  for (int first = 0; first < g.V; first += p.piece) {
    const int cols = std::min(p.piece, g.V - first);
    const Layout<T> beside{g.H, (const T*)g.x, dw != nullptr ? (T*)s.x : nullptr, (T*)dx, 0,
                           first == 0 ? std::min((g.T + 7) / 8, 256) : 0};
    const T* w = (const T*)g.w + first;
    LogitsArgs<T> a{{g.T, cols, g.x, g.H, w, g.V, s.list.rows}, g.H, s.list, tokens, own_list && first == 0};
    err = with_tile<T>(p.logits, [&](auto tile) {
      using C = decltype(tile);
      const bool tail = g.H % (kStageK<T> * C::KG) != 0;
      return tail ? run_dz<T, C, true>(a, first, p.piece, dz, beside, stream)
                  : run_dz<T, C, false>(a, first, p.piece, dz, beside, stream);
    });
    if (err != hipSuccess) return err;
    GradArgs b{};
    b.gx = TileSource{g.T, g.H, dz, p.piece, w, g.V, nullptr};
    b.gw = TileSource{g.H, dw != nullptr ? cols : 0, s.x, g.H, dz, p.piece, nullptr};
    b.Kx = dx != nullptr ? cols : 0;
    b.list = s.list;
    b.add = first > 0;
    b.sums = s.sums;
    b.dx = first + cols == g.V ? dx : nullptr;
    b.c = c;
    b.dw = dw != nullptr ? (T*)dw + first : nullptr;
    b.ldw = g.V;
    b.x_first = p.few || p.grads.x.each > p.grads.w.each;
    auto run = [&](auto tx, auto tw) {
      using CX = decltype(tx);
      using CW = decltype(tw);
      bm = CX::BM;
      slices.tiles = (g.T + bm - 1) / bm;
      b.slices = slices;
      b.nx = tiles_of<CX>(g.T, g.H) * slices.many;
      b.nw = dw != nullptr ? tiles_of<CW>(g.H, cols) : 0;
      constexpr int SX = kStageK<T> * CX::KG;
      const bool tail_x = cols % SX != 0 || slices.slice % SX != 0 || (slices.again && 128 % SX != 0);
      return tail_x ? run_grads<T, CX, CW, true>(b, stream) : run_grads<T, CX, CW, false>(b, stream);
    };
    const int pair = p.few ? -1 : p.grads.pair;
    err = hipErrorUnknown;
    if constexpr (sizeof(T) == 2) {
      if (p.few) err = run(DeepTile{}, DeepTile{});
      if (pair == 0) err = run(Tile0{}, Tile0{});
      if (pair == 1) err = run(Tile0{}, Tile1{});
      if (pair == 2) err = run(Tile1{}, Tile0{});
      if (pair == 3) err = run(Tile1{}, Tile1{});
    }
    if (pair == 4) err = run(Tile2{}, Tile2{});
    if (pair == 5) err = run(Tile3{}, Tile3{});
    if (pair == 6) err = run(Tile4<T>{}, Tile4<T>{});
    if (pair == 7) err = run(Tile5{}, Tile4<T>{});
    if (err != hipSuccess) return err;
  }
  if (!slices.again) return hipSuccess;
  const int64_t runs = (int64_t)g.T * (g.H / 8);
  MOE_LAUNCH(vocab_dx_kernel<T>, dim3((unsigned)std::min<int64_t>((runs + 255) / 256, 8192)), dim3(256), 0, stream, g.T, g.H,
             slices, bm, s.list, s.sums, c, (T*)dx);
  return hipGetLastError();
}

}  // namespace

size_t vocab_workspace_bytes(int T, int H, int V, int esize) {
  return remembered<size_t>(T, H, V, esize + 64, [&] {
    size_t need = vocab_space(nullptr, T, H, V, esize, vocab_plan(T, H, V, esize, false, false), false).bytes;
    for (int want = 1; want < 4; ++want)
      need = std::max(need, vocab_space(nullptr, T, H, V, esize, vocab_plan(T, H, V, esize, want & 1, want & 2), true).bytes);
    return need;
  });
}

hipError_t launch_vocab_fwd(const VocabArgs& g, int esize, float* loss, float* lse, float* mean, void* ws,
                            hipStream_t stream) {
  return esize == 4 ? vocab_fwd_typed<float>(g, loss, lse, mean, ws, stream)
                    : vocab_fwd_typed<uint16_t>(g, loss, lse, mean, ws, stream);
}

hipError_t launch_vocab_bwd(const VocabArgs& g, int esize, const float* loss, const float* lse, const float* mean,
                            const float* dloss, float scale, void* dx, void* dw, void* ws, hipStream_t stream) {
  return esize == 4 ? vocab_bwd_typed<float>(g, loss, lse, mean, dloss, scale, dx, dw, ws, stream)
                    : vocab_bwd_typed<uint16_t>(g, loss, lse, mean, dloss, scale, dx, dw, ws, stream);
}

}  // namespace moe
