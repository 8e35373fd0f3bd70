// moe_vocab_plan.h -- which workgroup tiles, pieces and slices run the products of
// moe_vocab.hip.  Host code only, a rule on sizes.
#pragma once

#include "moe_linear_plan.h"

namespace moe {

inline int rounded_up(int64_t v, int to) { return (int)((v + to - 1) / to * to); }

// Tiles of logits for few rows, beside those of moe_linear_plan.h: wide ones, whose stages hold 32 or 64 KiB of W, so
// that enough of it is on its way.  One forward over 2048 x 131072, us by rows:
//               1     64    128    192    256    320    384    512   1024
//   64 x 512    99     98    141    183    233    277    323    426    838
//   128 x 256   99    103    104    157    163    220    227    289    549
//   256 x 256  128    134    137    143    146    246    250    258    483
//   256 x 128  141    148    154    159    161    279    283    290    551
//   128 x 128 in two reduction groups, two stages   139 to 149 up to 128 rows
// and the dx products of one piece of 131072 columns on 128 x 128 tiles, frozen head, 128 rows: two groups of two
// stages 244 us the call, one of four 233.
enum { kTile64x512 = kTiles, kTile128x256 };
constexpr int kFewRows = 128;

struct VocabPlan {
  int logits;       // tile of the logits' products
  int piece;        // columns of a piece of the backward, a multiple of 512
  int pitch;        // rows of the statistics, of dz and of dx's sums
  bool few;         // the gradients' products on the tiles for few rows
  Plan2 grads;
};

// The columns of a piece: dz of 64 Mi elements, so that it is read again from the last-level cache, but at least 1024, so
// that the products keep their tiles.
constexpr int64_t kPieceElements = 64 << 20;

inline int64_t group_count(int M, int N, int bm, int bn) { return (int64_t)((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

inline int logits_tile(int T, int N, int H, int esize) {
  // the wide tiles where they fill the chip
  if (esize == 2 && T <= 64 && group_count(T, N, 64, 512) >= kCus / 2) return kTile64x512;
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
  p.few = esize == 2 && T <= kFewRows && group_count(H, p.piece, 128, 128) >= kCus;
  if (p.few && dx) {  // as many slices as fill the chip
    const int64_t slices = std::max<int64_t>(1, kCus / group_count(T, H, 128, 128));
    p.grads.x.slice = rounded_up((p.piece + slices - 1) / slices, 128);
    p.grads.x.slices = (p.piece + p.grads.x.slice - 1) / p.grads.x.slice;
  }
  return p;
}

}  // namespace moe
