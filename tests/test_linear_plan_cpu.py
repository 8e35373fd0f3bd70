"""The rule that picks tiles and reduction slices of the linear product
(csrc/moe_linear_plan.h, host code), compiled for the CPU: over many sizes every
slice holds some of the reduction, all but the last hold whole stages, together
they hold all of it, and the search always answers."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include "moe_linear_plan.h"
#include <cstdio>
#include <random>

static int bad = 0;
static void check(const moe::Cut& c, int M, int N, int K, int esize, const char* what) {
  const moe::TileCost& t = moe::cost_of(c.tile, esize);
  const long tiles = (long)((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
  bool ok = c.slices >= 1 && c.slices <= 16 && c.slice % 128 == 0 && (long)c.slices * c.slice >= K &&
            (long)(c.slices - 1) * c.slice < K && c.groups == tiles * c.slices && c.groups < (1l << 31);
  if (!ok && bad++ < 5) printf("%s M=%d N=%d K=%d: tile %d, %d slices of %d\n", what, M, N, K, c.tile, c.slices, c.slice);
}

int main() {
  std::mt19937 rng(1);
  auto log_size = [&](double lo, double hi) {
    return (int)std::exp(std::uniform_real_distribution<>(std::log(lo), std::log(hi))(rng));
  };
  for (int i = 0; i < 30000; ++i) {
    const int T = log_size(1, i % 10 ? 30000 : 1 << 30), I = 8 * log_size(1, i % 10 ? 2048 : 1 << 13), O = 8 * log_size(1, 2048);
    if ((long)T * std::max(I, O) >= 1l << 40) continue;  // refused
    for (int esize : {2, 4}) {
      check(moe::plan_fwd(T, O, I, esize), T, O, I, esize, "forward");
      for (int want = 1; want < 4; ++want) {
        const moe::Plan2 p = moe::plan_bwd(T, I, O, esize, want & 1, want & 2);
        if (want & 1) check(p.x, T, I, O, esize, "dx");
        if (want & 2) check(p.w, I, O, T, esize, "dw");
        const moe::Pair pair = moe::kPairs[p.pair];
        if (esize == 4 && p.pair < moe::kPairsF) ++bad;
        if (((want & 1) && pair.x != p.x.tile) || ((want & 2) && pair.w != p.w.tile)) ++bad;
      }
    }
  }
  return bad ? 1 : 0;
}
"""


def test_plans_cover_the_reduction(tmp_path):
    src = tmp_path / "plan.cpp"
    src.write_text("#include <cmath>\n" + SOURCE)
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "expert_grouped_gemm_top_amd", "csrc"), str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
