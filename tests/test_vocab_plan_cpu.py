"""The rule that picks the vocabulary loss' tiles, pieces and slices
(csrc/moe_vocab_plan.h, host code), compiled for the CPU: the sizes of
vocab_tile_cases.py still reach the kernels that they are there for, and over many
sizes pieces and slices cover the vocabulary."""
import os
import subprocess

import pytest

from vocab_tile_cases import CASES, TILES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
#include "moe_vocab_plan.h"

int main(int argc, char** argv) {
  for (int i = 1; i + 3 < argc; i += 4) {  // T H V and 1 dx + 2 dw
    const int T = atoi(argv[i]), H = atoi(argv[i + 1]), V = atoi(argv[i + 2]), want = atoi(argv[i + 3]);
    const moe::VocabPlan f = moe::make_vocab_plan(T, H, V, 2, false, false), p = moe::make_vocab_plan(T, H, V, 2, want & 1, want & 2);
    printf("%d %d %d %d %d %d\n", f.logits, p.logits, (V + p.piece - 1) / p.piece, p.few, p.grads.pair, p.grads.x.slices);
  }
  if (argc > 1) return 0;
  std::mt19937 rng(1);
  auto log_size = [&](double lo, double hi) {
    return (int)std::exp(std::uniform_real_distribution<>(std::log(lo), std::log(hi))(rng));
  };
  int bad = 0;
  for (int i = 0; i < 20000; ++i) {
    const int T = log_size(1, i % 10 ? 30000 : 1 << 24), H = 8 * log_size(1, 2048), V = 8 * log_size(1, 1 << 17);
    for (int esize : {2, 4})
      for (int want = 0; want < 4; ++want) {
        const moe::VocabPlan p = moe::make_vocab_plan(T, H, V, esize, want & 1, want & 2);
        const moe::Cut& x = p.grads.x;
        bool ok = p.pitch >= T && p.pitch % 256 == 0 && p.piece % 512 == 0 && p.piece > 0 && p.piece < V + 512;
        ok = ok && p.logits >= (esize == 2 ? 0 : (int)moe::kTile128x128) && (esize == 2 || p.logits < moe::kTiles);
        // pieces of dz hold 64 Mi elements, or the fewest columns
        ok = ok && ((int64_t)p.pitch * p.piece <= moe::kPieceElements || p.piece == 1024 || p.piece == moe::rounded_up(V, 512));
        if (want & 1) ok = ok && x.slice % 128 == 0 && x.slices >= 1 && (int64_t)x.slices * x.slice >= p.piece &&
                           (int64_t)(x.slices - 1) * x.slice < p.piece;
        if (!ok && bad++ < 5) printf("T=%d H=%d V=%d esize=%d want=%d\n", T, H, V, esize, want);
      }
  }
  return bad ? 1 : 0;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "expert_grouped_gemm_top_amd", "csrc"),
                    str(at / "plan.cpp"), "-o", str(at / "plan")], check=True)

    def run(*args):
        return subprocess.run([str(at / "plan"), *map(str, args)], capture_output=True, text=True)
    return run


def test_plans_cover_the_vocabulary(plan):
    r = plan()
    assert r.returncode == 0, r.stdout


def test_the_tile_cases_reach_their_kernels(plan):
    both, alone = (plan(*[v for c in CASES for v in (c.T, c.H, c.V, want)]).stdout.splitlines() for want in (3, 1))
    assert len(both) == len(alone) == len(CASES)
    for c, line, dx in zip(CASES, both, alone):
        loss, dz, pieces, few, pair, slices = map(int, line.split())
        bm, bn = TILES[c.loss]
        assert (loss, -(-c.T // bm) * -(-c.V // bn), dz, pieces, few, pair, slices, bool(int(dx.split()[3]))) == \
            (c.loss, c.tiles, c.loss, c.pieces, 0, c.pair, c.slices, c.few), c
    assert {c.loss for c in CASES if c.tiles > 256 and c.loss != 0} == {1, 6}  # every streamed tile, twice a workgroup
    assert {c.pair for c in CASES} >= {0, 1, 2, 3} and {c.pair for c in CASES if c.pieces > 1} >= {0, 1}
    assert sum(c.few for c in CASES) > 1


def choice(plan, T, H, V, want):
    """Tiles of the loss and of dz, and whether the products take the tiles for few rows."""
    loss, dz, _, few, _, _ = map(int, plan(T, H, V, want).stdout.split())
    return loss, dz, bool(few)


def test_few_rows_by_what_was_measured(plan):
    """The wide tile up to 128 rows and from 257 to 384 where it fills the chip, at vocabularies that divide over 256
    workgroups or not; the few-row tiles for dx alone, of 65 to 128 rows and long slices, never with dW beside it."""
    for H, V in ((2048, 131072), (2048, 151936), (4096, 151552), (2048, 65536)):
        for T in (1, 64, 65, 128, 257, 384):
            for want in (1, 2, 3):
                assert choice(plan, T, H, V, want) == (6, 6, want == 1 and 65 <= T <= 128 and V > 65536), (T, H, V, want)
        for T in (129, 256, 385, 512):
            assert choice(plan, T, H, V, 1)[0] != 6 and not choice(plan, T, H, V, 1)[2], (T, H, V)
    assert not choice(plan, 128, 1024, 32000, 1)[2]  # 32 slices of 1000 columns
