// moe_linear_plan.h -- which workgroup tiles and reduction slices run the
// products of moe_linear.hip.  Host code only, a rule on sizes: the plan of
// least estimated time, from the tiles' measured costs.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <iterator>

namespace moe {

// The workgroup tiles, largest first, and what a pass of them over the chip's
// 256 CUs takes: `step` us per 64 k (`step_few` when at most 160 workgroups
// run), `round` us for a tile's prologue and epilogue.  Measured on one MI355X with
// grids of 128, 256 and 512 workgroups and reductions of 512, 2048 and 4096
// (all three operand layouts within 8 %).  A larger tile moves fewer bytes
// through LDS per product (at 256 workgroups: 256 x 256 1.32 PFLOP/s,
// 256 x 128 1.14, 128 x 128 1.01, 128 x 64 0.84, 64 x 64 0.61) but leaves CUs
// idle where the outputs are few: 4099 x 768 over 2048 takes 49 us on 256 x 256,
// 30 on 256 x 128, 20.9 on 128 x 128, 25.8 on 128 x 64 tiles.
enum { kTile256x256 = 0, kTile256x128, kTile128x128, kTile128x64, kTile64x64, kTiles };
enum { kTileF128 = 0, kTileF64, kTilesF };
struct TileCost {
  int bm, bn;
  double step, step_few, round;
};
constexpr TileCost kCost[kTiles] = {{256, 256, 1.62, 1.18, 9.0},
                                    {256, 128, 0.94, 0.74, 5.0},
                                    {128, 128, 0.55, 0.47, 2.7},
                                    {128, 64, 0.35, 0.29, 2.1},
                                    {64, 64, 0.24, 0.20, 1.3}};
constexpr TileCost kCostF[kTilesF] = {{128, 128, 4.1, 4.05, 5.0}, {64, 64, 1.23, 1.22, 1.2}};  // fp32, per 64 k

constexpr int kCus = 256, kFew = 160;
constexpr double kLaunchUs = 3.5;           // one more kernel behind another
constexpr double kSliceBytesPerUs = 6.5e6;  // partials written and read again

inline const TileCost& cost_of(int tile, int esize) { return esize == 2 ? kCost[tile] : kCostF[tile]; }

// How a product is cut: its workgroup tile and the slices of its reduction.
struct Cut {
  int tile, slices, slice;  // k per slice
  int64_t groups;           // workgroups
  double each;              // us of one workgroup
  double after;             // us of adding the slices
};

inline Cut cut_of(int M, int N, int K, int esize, int tile, int want, bool few) {
  constexpr int kGrain = 128;  // slices are whole stages
  const TileCost& t = cost_of(tile, esize);
  Cut c{};
  c.tile = tile;
  c.slice = (int)((((int64_t)K + want - 1) / want + kGrain - 1) / kGrain * kGrain);
  c.slices = (K + c.slice - 1) / c.slice;
  c.groups = (int64_t)((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn) * c.slices;
  c.each = (double)((std::min(K, c.slice) + 63) / 64) * (few ? t.step_few : t.step) + t.round;
  c.after = c.slices > 1 ? (double)c.slices * M * N * 8.0 / kSliceBytesPerUs : 0.0;
  return c;
}

// Cuts worth a look: splitting a reduction pays where few tiles meet a long one
// (2048 x 768 outputs over 4099 rows: 56 us on 128 x 128 tiles, 31 us in two
// slices with the sum behind them).
template <typename Fn>
void each_cut(int M, int N, int K, int esize, int tile, Fn&& f) {
  int last = 0;
  for (int want : {1, 2, 3, 4, 6, 8, 12, 16}) {
    const Cut c = cut_of(M, N, K, esize, tile, want, false);
    if (want > 1 && c.groups > 2 * kCus) return;
    if (c.slices != last) f(c);
    last = c.slices;
  }
}

// The forward's cut of least estimated time: full passes over the CUs, then the rest.
inline Cut plan_fwd(int M, int N, int K, int esize) {
  Cut best{};
  double best_us = 0.0;
  for (int tile = 0; tile < (esize == 2 ? (int)kTiles : (int)kTilesF); ++tile)
    each_cut(M, N, K, esize, tile, [&](const Cut& c) {
      const int64_t rest = c.groups % kCus;
      double us = kLaunchUs + (double)(c.groups / kCus) * c.each + (c.slices > 1 ? kLaunchUs + c.after : 0.0);
      if (rest > 0) us += rest > kFew ? c.each : cut_of(M, N, K, esize, tile, c.slices, true).each;
      if (best.slices == 0 || us < best_us) {
        best = c;
        best_us = us;
      }
    });
  return best;
}

// The backward's cuts: dx and dw share a launch (Pairs: which tiles meet), so
// what counts is their joint work over the CUs, and the longest workgroup.
struct Plan2 {
  int pair;
  Cut x, w;
};
struct Pair {
  int x, w;
};
constexpr Pair kPairs[] = {{kTile256x256, kTile256x256}, {kTile256x256, kTile256x128}, {kTile256x128, kTile256x256},
                           {kTile256x128, kTile256x128}, {kTile128x128, kTile128x128}, {kTile128x64, kTile128x64},
                           {kTile64x64, kTile64x64}};
constexpr Pair kPairsF[] = {{kTileF128, kTileF128}, {kTileF64, kTileF64}};

inline Plan2 plan_bwd(int T, int I, int O, int esize, bool dx, bool dw) {
  Plan2 best{};
  double best_us = -1.0;
  const int pairs = esize == 2 ? (int)std::size(kPairs) : (int)std::size(kPairsF);
  for (int p = 0; p < pairs; ++p) {
    const Pair tiles = esize == 2 ? kPairs[p] : kPairsF[p];
    auto weigh = [&](const Cut* x, const Cut* w) {
      const int64_t gx = x ? x->groups : 0, gw = w ? w->groups : 0;
      const double ex = x ? x->each : 0.0, ew = w ? w->each : 0.0;
      double us = std::max({((double)gx * ex + (double)gw * ew) / kCus, ex, ew});
      if (gx + gw > kCus) us += 0.5 * std::min(gx ? ex : ew, gw ? ew : ex);  // the last ones end unevenly
      const double after = (x ? x->after : 0.0) + (w ? w->after : 0.0);
      if (after > 0.0) us += kLaunchUs + after;
      if (best_us < 0.0 || us < best_us) {
        best_us = us;
        best = Plan2{p, x ? *x : Cut{}, w ? *w : Cut{}};
      }
    };
    auto with_w = [&](const Cut* x) {
      if (!dw) return weigh(x, nullptr);
      each_cut(I, O, T, esize, tiles.w, [&](const Cut& w) { weigh(x, &w); });
    };
    if (!dx) with_w(nullptr);
    else each_cut(T, I, O, esize, tiles.x, [&](const Cut& x) { with_w(&x); });
  }
  return best;
}

}  // namespace moe
