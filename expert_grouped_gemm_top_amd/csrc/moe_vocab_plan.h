// moe_vocab_plan.h -- which workgroup tiles, pieces and slices run the products of
// moe_vocab.hip.  Host code only, a rule on sizes.
#pragma once

#include "moe_linear_plan.h"

namespace moe {

inline int rounded_up(int64_t v, int to) { return (int)((v + to - 1) / to * to); }

// The tile of logits for few rows, beside those of moe_linear_plan.h: a wide one, whose stages hold 32 KiB of W, so that
// enough of it is on its way.  One forward, us by rows:
//                          1     64    128    192    256    320    384    512
//   2048 x 131072
//     128 x 256          102    104    107    171    170    225    219    290
//     256 x 256          141    154    144    139    153    250    245    255
//     256 x 128          179    171    168    164    161    277    277    283
//   2048 x 151936
//     128 x 256          126    129    135    189    190    254    259    340
//     256 x 256          173    176    176    182    186    287    299    300
//     256 x 128          169    171    180    185    186    331    334    338
//   4096 x 151552
//     128 x 256          239    247    254    341    350    481    478    645
//     256 x 256          322    328    335    335    347    545    549    565
//   2048 x 65536
//     128 x 256           57     59     59     83     84    120    115    149
//     256 x 256           69     74     76     75     74    133    127    136
//   1024 x 32000 (125 tiles a row of them: the estimate decides)
//     128 x 256           27     30     30     32     33     48     48     51
//     256 x 256           35     38     39     39     41     44     45     46
// (A 64 x 512 tile took 100 us where 128 x 256 takes 102 at one row of 131072 columns, 153 against 126 at 151936.)
enum { kTile128x256 = kTiles };

struct VocabPlan {
  int logits;       // tile of the logits' products
  int piece;        // columns of a piece of the backward, a multiple of 512
  int pitch;        // rows of the statistics, of dz and of dx's sums
  bool few;         // dx's products on the tiles for few rows
  Plan2 grads;
};

// The columns of a piece: dz of 64 Mi elements, so that it is read again from the last-level cache, but at least 1024, so
// that the products keep their tiles.
constexpr int64_t kPieceElements = 64 << 20;

inline int64_t group_count(int M, int N, int bm, int bn) { return (int64_t)((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

inline int logits_tile(int T, int N, int H, int esize) {
  // the wide tile where it fills the chip
  if (esize == 2 && group_count(T, N, 128, 256) >= kCus && (T <= 128 || (T > 256 && T <= 384))) return kTile128x256;
  int best_tile = 0;
  double best = -1.0;
  for (int tile = esize == 2 ? 0 : (int)kTile128x128; tile < kTiles; ++tile) {
    const Cut c = cut_of(T, N, H, esize, tile, 1);
    const int64_t rest = c.groups % kCus;
    double us = (double)(c.groups / kCus) * c.each;
    if (rest > 0) us += pass_us(cost_of(tile, esize), H, rest);
    if (best < 0.0 || us < best) {
      best = us;
      best_tile = tile;
    }
  }
  return best_tile;
}

inline VocabPlan make_vocab_plan(int T, int H, int V, int esize, bool dx, bool dw) {
  VocabPlan p{};
  p.pitch = rounded_up(T, 256);
  const int64_t cols = std::max<int64_t>(kPieceElements / p.pitch / 512 * 512, 1024);
  p.piece = (int)std::min<int64_t>(cols, rounded_up(V, 512));
  p.logits = logits_tile(T, dx || dw ? p.piece : V, H, esize);
  if (!dx && !dw) return p;
  p.grads = plan_bwd(T, H, p.piece, esize, dx, dw, false);
  // dx alone, of 65 to 128 rows: 128 x 128 tiles in one reduction group of four stages and as many slices as fill the
  // chip, where those are long.  The call with and without, us: 128 rows, 2048 x 131072 (slices of 8192) 242 and 260,
  // 2048 x 151936 289 and 303, 4096 x 151552 529 and 561, 2048 x 65536 (4096) 142 and 142, 1024 x 32000 (1024) 56 and 52;
  // 64 rows of 2048 x 131072 215 and 210; with dW beside it 600 and 490.
  const int64_t slices = std::max<int64_t>(1, kCus / group_count(T, H, 128, 128));
  const int slice = rounded_up((p.piece + slices - 1) / slices, 128);
  p.few = esize == 2 && dx && !dw && T > 64 && T <= 128 && slice >= 8192;
  if (p.few) {
    p.grads.x.slice = slice;
    p.grads.x.slices = (p.piece + slice - 1) / slice;
  }
  return p;
}

}  // namespace moe
