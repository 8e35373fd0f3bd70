// moe_linear_plan.h -- which workgroup tiles and reduction slices run the
// products of moe_linear.hip.  Host code only, a rule on sizes: the plan of
// least estimated time, from the tiles' measured costs.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <iterator>

namespace moe {

// The workgroup tiles, largest first, and what a pass of them over the chip's
// 256 CUs takes: `step` us per 64 k (`step_few` when at most 128 workgroups
// run), `round` us for a tile's prologue and epilogue.  Measured on one MI355X with
// grids of 128, 256 and 512 workgroups and reductions of 512 to 8192 (all three
// operand layouts within 8 %), the small tiles' a little up where many of them
// run.  A larger tile moves fewer bytes
// through LDS per product (at 256 workgroups: 256 x 256 1.31 PFLOP/s,
// 256 x 128 1.13, 128 x 128 0.99, 128 x 64 0.75, 64 x 64 0.61) but leaves CUs
// idle where the outputs are few: 4099 x 768 over 2048 takes 48 us on 256 x 256,
// 30 on 256 x 128, 21 on 128 x 128, 27 on 128 x 64 tiles.  32 x 32 is for a few
// rows, where the weights' way through as many CUs as there are is what counts.
enum { kTile256x256 = 0, kTile256x128, kTile128x128, kTile128x64, kTile64x64, kTile32x32, kTiles };
struct TileCost {
  int bm, bn;
  double step, step_few, round;
};
constexpr TileCost kCost[kTiles] = {{256, 256, 1.64, 1.12, 9.5},
                                    {256, 128, 0.95, 0.70, 5.5},
                                    {128, 128, 0.54, 0.43, 3.5},
                                    {128, 64, 0.37, 0.29, 2.5},
                                    {64, 64, 0.26, 0.20, 2.0},
                                    {32, 32, 0.18, 0.14, 2.0}};
// fp32, which takes the last four (256 workgroups: 138, 128, 120 and 95 TFLOP/s).
constexpr TileCost kCostF[kTiles] = {{},
                                     {},
                                     {128, 128, 3.9, 3.9, 6.5},
                                     {128, 64, 2.1, 2.1, 4.0},
                                     {64, 64, 1.12, 1.12, 1.2},
                                     {32, 32, 0.40, 0.31, 2.5}};

constexpr int kCus = 256;
constexpr double kLaunchUs = 4.5;           // one more kernel behind another
constexpr double kSliceBytesPerUs = 6.5e6;  // partials written and read again

inline const TileCost& cost_of(int tile, int esize) { return esize == 2 ? kCost[tile] : kCostF[tile]; }

// How a product is cut: its workgroup tile and the slices of its reduction.
struct Cut {
  int tile, slices, slice;  // k per slice
  int64_t groups;           // workgroups
  double each;              // us of one workgroup
  double after;             // us of adding the slices
};

// us of a pass of `groups` workgroups (at most 256) over reductions of k.
inline double pass_us(const TileCost& t, int k, int64_t groups) {
  const double least = t.bm == 32 ? -0.5 : 0.0;  // the smallest tile's step falls on down to 64 workgroups
  const double full = std::min(std::max((double)(groups - 128) / 128.0, least), 1.0);
  return (double)((k + 63) / 64) * (t.step_few + full * (t.step - t.step_few)) + t.round;
}

inline Cut cut_of(int M, int N, int K, int esize, int tile, int want) {
  // Whole stages of all tiles but the smallest, whose eight reduction groups take
  // 512 k (fp32: 256) to a stage: a slice may end inside one of its stages, the
  // rest of which is masked, and the estimate counts the k that are there.
  constexpr int kGrain = 128;
  const TileCost& t = cost_of(tile, esize);
  Cut c{};
  c.tile = tile;
  c.slice = (int)((((int64_t)K + want - 1) / want + kGrain - 1) / kGrain * kGrain);
  c.slices = (K + c.slice - 1) / c.slice;
  c.groups = (int64_t)((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn) * c.slices;
  c.each = pass_us(t, std::min(K, c.slice), kCus);
  c.after = c.slices > 1 ? (double)c.slices * M * N * 8.0 / kSliceBytesPerUs : 0.0;
  return c;
}

// Cuts worth a look: splitting a reduction pays where few tiles meet a long one
// (2048 x 768 outputs over 4099 rows: 38 us on 128 x 128 tiles, 30 us in two
// slices with the sum behind them).
template <typename Fn>
void each_cut(int M, int N, int K, int esize, int tile, Fn&& f) {
  int last = 0;
  for (int want : {1, 2, 3, 4, 6, 8, 12, 16}) {
    const Cut c = cut_of(M, N, K, esize, tile, want);
    if (want > 1 && c.groups > 2 * kCus) return;
    if (c.slices != last) f(c);
    last = c.slices;
  }
}

// The forward's cut of least estimated time: full passes over the CUs, then the rest.
inline Cut plan_fwd(int M, int N, int K, int esize) {
  Cut best{};
  double best_us = 0.0;
  for (int tile = esize == 2 ? 0 : (int)kTile128x128; tile < kTiles; ++tile)
    each_cut(M, N, K, esize, tile, [&](const Cut& c) {
      const int64_t rest = c.groups % kCus;
      double us = kLaunchUs + (double)(c.groups / kCus) * c.each + (c.slices > 1 ? kLaunchUs + c.after : 0.0);
      if (rest > 0) us += pass_us(cost_of(tile, esize), std::min(K, c.slice), rest);
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
                           {kTile64x64, kTile64x64}, {kTile32x32, kTile64x64}};
constexpr int kPairsF = 4;  // fp32 takes those from here on

inline Plan2 plan_bwd(int T, int I, int O, int esize, bool dx, bool dw) {
  Plan2 best{};
  double best_us = -1.0;
  for (int p = esize == 2 ? 0 : kPairsF; p < (int)std::size(kPairs); ++p) {
    const Pair tiles = kPairs[p];
    auto weigh = [&](const Cut* x, const Cut* w) {
      const int64_t gx = x ? x->groups : 0, gw = w ? w->groups : 0;
      const int64_t load = std::min<int64_t>(gx + gw, kCus);
      const double ex = x ? pass_us(cost_of(tiles.x, esize), std::min(O, x->slice), load) : 0.0;
      const double ew = w ? pass_us(cost_of(tiles.w, esize), std::min(T, w->slice), load) : 0.0;
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
