"""The vocabulary loss on its main kernels (vocab_tile_cases.py has the sizes): every
streamed tile with workgroups that take a second one, and the gradients' large tiles
over one and several pieces, against the 64-bit formula on the device, with tokens
that are not counted, NaN in their rows, and padding columns."""
import math

import pytest
import torch

from block_ref import U
from expert_grouped_gemm_top_amd import moe
from moe_cases import note
from test_gpu_vocab import Buffers
from vocab_tile_cases import CASES

pytestmark = pytest.mark.gpu


def inputs(T, H, V, vocab, seed):
    """Values of few bits, so that fp32 holds every logit exactly in any order of its sum; logits of a deviation near 3,
    so that a row's probability lies on a few classes, others in each row.  A third of the targets are the likeliest class."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    whole = lambda most, *s: torch.randint(-most, most + 1, s, generator=g, device="cuda").double()  # noqa: E731
    x = whole(2, T, H)
    w = whole(8, H, V) * 2.0 ** -round(math.log(H * 48 / 9, 4))
    assert float((x.abs() @ w.abs()).max()) < 2 ** 11  # multiples of 2^-7 and more: below 2^24 of them
    y = torch.randint(0, vocab, (T,), generator=g, device="cuda", dtype=torch.int32)
    y[::3] = (x[::3] @ w[:, :vocab].contiguous()).argmax(1).int()
    y[torch.rand(T, generator=g, device="cuda") < 0.3] = -100
    y[:2] = torch.tensor([vocab - 1, 0])  # one at least in the last columns
    return x, w, y


def reference(x, w, y, vocab, dloss, scale):
    keep = y >= 0
    rows = torch.nonzero(keep)[:, 0]
    n = len(rows)
    wv = w[:, :vocab].contiguous()
    l = x[rows] @ wv
    at = torch.arange(n, device="cuda"), y[rows].long()
    lse, own = torch.logsumexp(l, 1), l[at]
    p = torch.exp(l - lse[:, None])
    p[at] -= 1
    p *= scale * (torch.full((n,), 1.0 / n, dtype=torch.float64, device="cuda") if dloss is None else dloss[rows].double())[:, None]
    out = dict(rows=rows, n=n, lse=lse, loss=lse - own, most=l.abs().amax(1))
    out.update(dx=p @ wv.t().contiguous(), dw=x[rows].t().contiguous() @ p)
    p.abs_(), wv.abs_()
    out.update(sx=p @ wv.t().contiguous(), sw=x[rows].abs().t().contiguous() @ p)
    return out


def over(got, want, bound):
    return float(((got.double() - want).abs() - bound).max())


# The logits are exact.  A statistic is off by its exponentials' and logarithms' roundings, (|lse| + |logit| + 64) 2^-23,
# and its additions: at most 128 columns a lane, the lanes and waves of a run, 64 of the runs at a time, 2^-24 each.  The
# others' softmax goes by lse and the loss' logarithm, their probability by the loss: three times that.
@pytest.mark.parametrize("dx,dw", [(True, True), (True, False)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c.T}x{c.H}x{c.V}")
def test_tiles(case, dx, dw):
    T, H, V = case.T, case.H, case.V
    vocab, weighted = V - 3, T % 2 == 0
    note(f"vocab tiles T={T} H={H} V={V} dx={dx} dw={dw}")
    x, w, y = inputs(T, H, V, vocab, T + H)
    dloss = torch.rand(T, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") if weighted else None
    b = Buffers(T, H, V, "bf16", dx, dw)
    spoiled = x.clone()
    spoiled[y < 0] = float("nan")
    b.step(spoiled.bfloat16(), w.bfloat16(), y, vocab, dloss, 0.5)
    torch.cuda.synchronize()
    r = reference(x, w, y, vocab, dloss, 0.5)
    rows, u = r["rows"], U["bf16"]
    off = (r["lse"].abs() + r["most"] + 64) * 2.0 ** -23 + (256 + V / 8192) * 2.0 ** -24
    assert over(b.lse[rows], r["lse"], off + U["f32"] * r["lse"].abs()) <= 0
    assert over(b.loss[rows], r["loss"], off + U["f32"] * r["loss"].abs()) <= 0
    assert abs(float(b.mean[0]) - float(r["loss"].mean())) <= float(off.max()) + 2 * U["f32"] * float(r["loss"].mean())
    assert abs(float(b.mean[1]) - 1 / r["n"]) <= U["f32"] / r["n"]
    rel = 3 * float(off.max()) + 16 * 2.0 ** -23
    others = torch.nonzero(y < 0)[:, 0]
    assert (b.loss[others] == 0).all() and (b.lse[others] == 0).all()
    if dx:
        assert over(b.dx[rows], r["dx"], (rel + u + vocab * 2.0 ** -23) * r["sx"] + u * r["dx"].abs() + 1e-38) <= 0
        assert (b.dx[others] == 0).all()
    if dw:  # q - [v = y] and the rows of x times f are rounded
        assert over(b.dw[:, :vocab], r["dw"], (rel + 2 * u + u * u + r["n"] * 2.0 ** -23) * r["sw"] + u * r["dw"].abs() + 1e-38) <= 0
        assert (b.dw[:, vocab:] == 0).all()


def test_a_second_tile_under_captured_replays():
    """Streamed tiles replayed with other inputs and other counted tokens: as the eager calls, bit for bit."""
    T, H, V = 100, 64, 70000
    x, w, y = inputs(T, H, V, V, 5)
    x, w = x.bfloat16(), w.bfloat16()
    a, e = Buffers(T, H, V, "bf16"), Buffers(T, H, V, "bf16")
    a.step(x, w, y, V)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step(x, w, y, V)
    for i in range(4):
        nx, nw, ny = inputs(T, H, V, V, 30 + i)
        x.copy_(nx), w.copy_(nw), y.copy_(ny)
        for t in a.outputs():
            t.fill_(3)
        g.replay()
        e.step(x, w, y, V)
        torch.cuda.synchronize()
        for p, q in zip(a.outputs(), e.outputs()):
            assert torch.equal(p, q), i


def test_launches_of_a_streamed_call():
    x, w, y = inputs(100, 64, 70000, 70000, 6)
    b = Buffers(100, 64, 70000, "bf16")
    before = moe.moe_launch_count()
    b.step(x.bfloat16(), w.bfloat16(), y, 70000)
    assert moe.moe_launch_count() - before == 2 + 2 + 1  # dx is cut into slices
