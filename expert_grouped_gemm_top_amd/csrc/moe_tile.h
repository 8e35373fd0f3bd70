// moe_tile.h -- one workgroup tile of a dense product on the matrix cores, for
// the products of moe_linear.hip and moe_vocab.hip: operands of either layout
// by direct loads into LDS, bf16 on 32x32x16 and fp32 on 32x32x2, the outputs
// handed on in runs of eight.
#pragma once

#include <type_traits>

#include "moe_common.h"
#include "moe_lds32.h"

namespace moe {

// Operands of C [M, N] = A B.  Either may lie with k contiguous ("KC":
// a[m lda + k], b[n ldb + k]) or with its own index contiguous (a[k lda + m],
// b[k ldb + n]).  rows: row m of a KC operand a is its row rows[m].
struct TileSource {
  int M, N;
  const void* a;
  int64_t lda;
  const void* b;
  int64_t ldb;
  const int32_t* rows;
};

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
  __device__ void init(const void* base, int64_t ld, const int32_t* map, int r0, int rows, int k0, int stage_k, int w,
                       int l) {
    step = KC ? stage_k : stage_k * ld;
#pragma unroll
    for (int i = 0; i < INS; ++i) {
      if (KC) {
        const int row = 8 * (INS * w + i) + l / 8;
        k[i] = k0 + CH * kc_key(row, l % 8);
        int r = min(r0 + row, rows - 1);
        if (map != nullptr) r = map[r];
        src[i] = (const T*)base + (int64_t)r * ld + k[i];
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
  // columns that leave at a time, as the stage buffers hold them in fp32
  static constexpr int FIT = LDS / (BM * 4), OUT_COLS = FIT >= BN ? BN : (FIT >= 128 ? 128 : 64);
};
constexpr int kTileThreads = 512;

// A tile's sums as bf16 rows: make(row, col, v) turns four neighbouring sums (row and
// column of the tile) into the values to store, put(row, col, q) stores eight of
// them.  They change places in LDS, [row][BN] with 16-byte chunk c of row r at
// c ^ (r mod 16), so that whole 16-byte lanes of contiguous row runs leave.
template <typename C, int MI, int NJ, typename Make, typename Put>
__device__ __forceinline__ void leave_bf16(f32x16 (&acc)[MI][NJ], unsigned char* s_dyn, Make&& make, Put&& put) {
  constexpr int BM = C::BM, BN = C::BN, CH = BN / 8, KEY = CH < 16 ? CH - 1 : 15;
  static_assert(C::KG == 1 && BM * BN * 2 <= C::LDS, "staging");
  const int tid = threadIdx.x, l32 = tid & 31, hk = (tid >> 5) & 1, w = tid >> 6;
  const int row0 = BM / C::WM * (w % C::WM) + l32, col0 = BN / (C::NW / C::WM) * (w / C::WM) + 4 * hk;
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = row0 + 32 * i, col = col0 + 32 * j + 8 * q;
        float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        make(i, row, col, v);
        *(u32x2*)(s_dyn + row * (2 * BN) + 16 * ((col >> 3) ^ (row & KEY)) + 2 * (col & 7)) =
            u32x2{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3])};
      }
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the staged values are written
  barrier_no_fence();
#pragma unroll 4
  for (int it = tid; it < BM * CH; it += 64 * C::NW) {
    const int row = it / CH, c = it % CH;
    put(row, 8 * c, *(const u32x4*)(s_dyn + row * (2 * BN) + 16 * (c ^ (row & KEY))));
  }
}

// The same without LDS, for stage buffers that are being loaded: the two lanes of a row exchange their halves, and each
// leaves every other 16-byte run.
template <typename C, int MI, int NJ, typename Make, typename Put>
__device__ __forceinline__ void leave_bf16_direct(f32x16 (&acc)[MI][NJ], Make&& make, Put&& put) {
  const int tid = threadIdx.x, l32 = tid & 31, hk = (tid >> 5) & 1, w = tid >> 6;
  const int row0 = C::BM / C::WM * (w % C::WM) + l32, col0 = C::BN / (C::NW / C::WM) * (w / C::WM);
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        const int row = row0 + 32 * i, col = col0 + 32 * j + 8 * q;
        uint32_t half[2][2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float v[4] = {acc[i][j][4 * (q + p)], acc[i][j][4 * (q + p) + 1], acc[i][j][4 * (q + p) + 2],
                        acc[i][j][4 * (q + p) + 3]};
          make(i, row, col + 8 * p + 4 * hk, v);
          half[p][0] = pack_bf2(v[0], v[1]);
          half[p][1] = pack_bf2(v[2], v[3]);
        }
        // lanes 32 to 63 of run q change places with lanes 0 to 31 of run q + 1
        const auto a = __builtin_amdgcn_permlane32_swap(half[0][0], half[1][0], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(half[0][1], half[1][1], false, false);
        put(row, col + 8 * hk, u32x4{a[0], b[0], a[1], b[1]});
      }
}

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

// Output tiles over k in [kb, ke), none where kb == ke, one after the other: `next`
// gives them, next(mt, nt), until it says that there are no more.  A stage
// is waited for before the last run of the one in front, so its first
// fragments are read under those products, and its successor's loads go out in
// two halves before the next two runs of products.
// `out` gets the outputs.  Where Out::kWhole (tiles of one reduction group), out.tile
// gets the sums as they lie in the waves' registers, with the stage buffers free:
// register r of acc[i][j] is row TM wm + 32 i + l32 of the tile, column
// TN wn + 32 j + 8 (r / 4) + 4 hk + r % 4.  STREAM, for an out.tile that leaves
// the stage buffers alone: the next tile's first stages load meanwhile, and what it
// needs from memory out.ahead has put into LDS before the tile's products (behind a
// barrier of the last out.tile), so that no wait for that waits for those loads.  Else out.skip(m, n) says that a run is not wanted, and
// out(m, n, v, lanes) takes the eight outputs of row m from column n on; `lanes`
// neighbouring lanes, a constant, hold 8 lanes neighbouring columns of a row.
template <typename T, bool AKC, bool BKC, typename C, bool TAIL, bool STREAM, typename Next, typename Out>
__device__ __forceinline__ void tile_products(const TileSource& g, Next&& next, int kb, int ke, unsigned char* s_dyn,
                                              Out&& out) {
  constexpr int BM = C::BM, BN = C::BN, NW = C::NW, WM = C::WM, KG = C::KG, STAGES = C::STAGES;
  constexpr int BK = kStageK<T>, RUN = kRunProducts<T>;
  constexpr int TM = BM / WM, TN = BN / (NW / WM), MI = TM / 32, NJ = TN / 32;
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, GROUP = A_BYTES + B_BYTES, STAGE = KG * GROUP;
  const int tid = threadIdx.x, l = tid & 63, l32 = l & 31, hk = l >> 5;
  const int kg = (tid >> 6) / NW, w = (tid >> 6) % NW;
  const int wm = w % WM, wn = w / WM;
  static_assert(!STREAM || std::remove_reference_t<Out>::template kWhole<C>, "no stage buffer for the outputs");
  const int steps = (ke - kb + KG * BK - 1) / (KG * BK);
  int mt, nt;
  if (!next(mt, nt)) return;
  int m0 = mt * BM, n0 = nt * BN;

  Loader<T, AKC, BM, NW, TAIL> la;
  Loader<T, BKC, BN, NW, TAIL> lb;
  constexpr int INS = Loader<T, AKC, BM, NW, TAIL>::INS + Loader<T, BKC, BN, NW, TAIL>::INS;  // loads of a stage
  // stage s lies in buffer s % STAGES; a group loads and reads its own part of it
  unsigned char* const mine = s_dyn + kg * GROUP;
  auto issue_a = [&](int buf) { la.issue(ke, KG * BK, mine + buf * STAGE, w); };
  auto issue_b = [&](int buf) { lb.issue(ke, KG * BK, mine + buf * STAGE + A_BYTES, w); };

  // the first stages of tile (m0, n0)
  auto start = [&] {
    la.init(g.a, g.lda, g.rows, m0, g.M, kb + kg * BK, KG * BK, w, l);
    lb.init(g.b, g.ldb, nullptr, n0, g.N, kb + kg * BK, KG * BK, w, l);
    for (int s = 0; s < STAGES - 1 && s < steps; ++s) {
      issue_a(s);
      issue_b(s);
    }
  };
  start();

  f32x16 acc[MI][NJ];
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

next_tile:
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  if constexpr (STREAM) out.template ahead<C>(m0);
  if (steps > 0) {
    Frags f0, f1;
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
  }

  if constexpr (std::remove_reference_t<Out>::template kWhole<C>) {
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's last fragment reads are done
    barrier_no_fence();                   // ... and every wave's
    if constexpr (STREAM) {
      const int m = m0, n = n0;
      const bool more = next(mt, nt);
      if (more) {
        m0 = mt * BM;
        n0 = nt * BN;
        start();
      }
      out.template tile<C>(acc, m, n, s_dyn);
      if (more) goto next_tile;
    } else {
      out.template tile<C>(acc, m0, n0, s_dyn);
    }
    return;
  }
  // The fp32 tile leaves through the idle stage buffers, HC columns at a time
  // ([row][HC], 16-byte chunk c of row r at c ^ (r mod CH)), so that the epilogue
  // reads and writes runs of eight neighbouring outputs.
  constexpr int FIT = C::FIT, HC = C::OUT_COLS;
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
      if (out.skip(m, n)) continue;
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
      out(m, n, v, std::integral_constant<int, HC / 8>{});
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's reads of the staged rows are done
  }
}

// One output tile.
template <typename T, bool AKC, bool BKC, typename C, bool TAIL, typename Out>
__device__ __forceinline__ void tile_product(const TileSource& g, int mt, int nt, int kb, int ke, unsigned char* s_dyn,
                                             Out&& out) {
  auto once = [&](int& m, int& n) {
    m = mt;
    n = nt;
    return true;
  };
  tile_products<T, AKC, BKC, C, TAIL, false>(g, once, kb, ke, s_dyn, out);
}

}  // namespace moe
