"""GPU parity of routing by scores (moe_route_scored, moe_route_scored_bwd and
moe_router_bwd_dlogits) against the 64-bit references of block_ref.py: choices
bit for bit, weights and gradients within bounds counted from the formulas."""
import numpy as np
import pytest
import torch

import block_ref as R
from expert_grouped_gemm_top_amd import moe
from moe_cases import note

pytestmark = pytest.mark.gpu

INF = float("inf")


def run(l, bias, k, score, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    T, E = l.shape
    note(f"route T={T} E={E} k={k} score={score} bias={bias is not None} groups={groups},{top_groups},{group_top} "
         f"renorm={renorm}")
    ld = torch.from_numpy(np.ascontiguousarray(l, np.float32)).cuda()
    bd = None if bias is None else torch.from_numpy(np.ascontiguousarray(bias, np.float32)).cuda()
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    moe.moe_route_scored(ld, bd, idx, w, k, score, groups, top_groups, group_top, renorm, scale)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), R.host(w)


def weight_bound(l, idx, ref, scale):
    """fp32 steps of a weight: the log score (its terms |l| + 1, three roundings each), the difference to
    the largest, exp and its argument (2^-24 per unit of the argument), the sum of k <= 16 terms, the quotient and
    the scale -- at most 8 (|l|max + 4) + 16 half steps; 2^-140 where fp32 has no normal numbers."""
    sel = np.take_along_axis(np.where(np.isfinite(l), np.abs(l), 0), idx, axis=1).max(1, keepdims=True)
    top = np.where(np.isfinite(l), np.abs(l), 0).max(1, keepdims=True)
    return (8 * (np.maximum(sel, top) + 4) + 16) * 2.0 ** -24 * np.abs(ref) + abs(scale) * 2.0 ** -140


def check(l, bias, k, score, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    l = np.asarray(l, np.float32).astype(np.float64)
    bias = None if bias is None else np.asarray(bias, np.float32).astype(np.float64)
    ri, rw = R.route(l, bias, k, score, groups, top_groups, group_top, renorm, scale)
    gi, gw = run(l, bias, k, score, groups, top_groups, group_top, renorm, scale)
    bad = np.nonzero((ri != gi).any(1))[0]
    if len(bad):  # only where the sums tie as real numbers and their rounding decides
        open_ = R.undecided(l[bad], bias, k, score, groups, top_groups, group_top)
        wrong = bad[~open_]
        assert not len(wrong), f"token {wrong[0]} of {len(wrong)}: {gi[wrong[0]]} for {ri[wrong[0]]}"
        rw[bad] = R.weights(l[bad], gi[bad], score, renorm, scale)
    R.within("topk_w", gw, rw, weight_bound(l, gi, rw, scale))


SHAPES = [  # T, E, k, groups, top_groups
    (1, 1, 1, 1, 1), (3, 2, 2, 2, 2), (5, 8, 2, 4, 2), (33, 16, 4, 4, 1), (17, 17, 3, 1, 1), (64, 37, 16, 1, 1),
    (9, 64, 8, 16, 3), (130, 100, 7, 5, 2), (257, 128, 8, 8, 4), (100, 160, 6, 8, 3), (31, 200, 16, 10, 2),
    (515, 256, 8, 8, 4), (16, 256, 16, 16, 1), (12, 241, 1, 1, 1), (40, 48, 5, 3, 2), (7, 90, 9, 9, 1),
]


@pytest.mark.parametrize("T,E,k,groups,top_groups", SHAPES)
@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
def test_route_matches_reference(T, E, k, groups, top_groups, score):
    rng = np.random.default_rng(T * 1000 + E)
    l = rng.standard_normal((T, E)) * 1.5
    bias = 0.1 * rng.standard_normal(E)
    for b in (None, bias):
        for renorm, scale in ((True, 2.5), (False, 1.0)):
            check(l, b, k, score, renorm=renorm, scale=scale)
            if groups > 1:
                for group_top in (1, 2)[:E // groups]:
                    check(l, b, k, score, groups, top_groups, group_top, renorm, scale)


def test_route_large_batch():
    rng = np.random.default_rng(11)
    l = rng.standard_normal((16384, 256))
    bias = 0.05 * rng.standard_normal(256)
    check(l, bias, 8, R.SIGMOID, 8, 4, 2, True, 2.5)
    check(l[:, :128], None, 8, R.SOFTMAX)
    check(l[:, :128], bias[:128], 8, R.SOFTMAX, renorm=False)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
def test_route_ties_go_to_the_lower_index(score):
    """Logits on a grid of a quarter: exact ties inside and across groups."""
    rng = np.random.default_rng(5)
    l = np.round(rng.standard_normal((300, 128)) * 4) / 4
    for b in (None, np.zeros(128), np.repeat([0.25, 0.0, 0.5, 0.25], 32)):
        check(l, b, 8, score)
        check(l, b, 8, score, 8, 2, 1)
        check(l, b, 8, score, 8, 2, 2)
    check(np.zeros((5, 128)), None, 8, score, 8, 2, 2)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("E,k,groups,top_groups", [(256, 16, 16, 4), (60, 16, 6, 3), (60, 5, 6, 3), (16, 16, 4, 4), (13, 12, 1, 1)])
def test_route_ties_of_long_lists_and_odd_groups(score, E, k, groups, top_groups):
    rng = np.random.default_rng(E + k)
    for grid in (4.0, 64.0):  # many ties, and some
        l = np.round(rng.standard_normal((120, E)) * grid) / grid
        for b in (None, np.zeros(E), np.round(rng.standard_normal(E) * 4) / 16):
            check(l, b, k, score)
            for group_top in (1, 2):
                check(l, b, k, score, groups, top_groups, group_top)


def test_route_of_tensors_off_the_alignment():
    """Rows and bias that start at any multiple of four bytes."""
    rng = np.random.default_rng(13)
    T, E, k = 70, 128, 8
    for shift in (1, 2, 3):
        note(f"route shifted by {shift}")
        flat = torch.from_numpy(np.float32(rng.standard_normal(T * E + E + 8))).cuda()
        l, b = flat[shift:shift + T * E].view(T, E), flat[T * E + 4 - shift:T * E + 4 - shift + E]
        out = torch.zeros(2 * T * k + 4, device="cuda")
        w = out[shift:shift + T * k].view(T, k)
        idx = torch.zeros(T * k + 4, dtype=torch.int32, device="cuda")[shift:shift + T * k].view(T, k)
        moe.moe_route_scored(l, b, idx, w, k, R.SIGMOID, 8, 4, 2, True, 1.0)
        d = torch.zeros(T * E + 4, device="cuda")[shift:shift + T * E].view(T, E)
        moe.moe_route_scored_bwd(l, idx, w, d, R.SOFTMAX, False)
        torch.cuda.synchronize()
        ri, rw = R.route(R.host(l), R.host(b), k, R.SIGMOID, 8, 4, 2)
        assert np.array_equal(idx.cpu().numpy(), ri)
        R.within("topk_w", R.host(w), rw, weight_bound(R.host(l), ri, rw, 1.0))
        ref = R.route_bwd(R.host(l), ri, R.host(w), R.SOFTMAX, False, 1.0)
        R.within("dlogits", R.host(d), ref, 400 * 2.0 ** -24)  # as in check_bwd: E = 128, weights below 1


def test_route_rows_past_32_bits():
    """More than 2^31 logits: the last tokens, and the first."""
    T, E, k = (1 << 31) // 256 + 1000, 256, 4
    note(f"route T={T} E={E}")
    l = torch.zeros(T, E, device="cuda")
    rng = np.random.default_rng(14)
    some = np.float32(rng.standard_normal((500, E)))
    l[:500], l[-500:] = torch.from_numpy(some).cuda(), torch.from_numpy(some).cuda()
    idx, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    moe.moe_route_scored(l, None, idx, w, k, R.SIGMOID)
    d = torch.full((T, E), 7.0, device="cuda")
    moe.moe_route_scored_bwd(l, idx, w, d, R.SIGMOID)
    torch.cuda.synchronize()
    ri, rw = R.route(some, None, k, R.SIGMOID)
    ref = R.route_bwd(some, ri, np.float32(rw), R.SIGMOID, True, 1.0)
    for rows in (slice(0, 500), slice(T - 500, T)):
        assert np.array_equal(idx[rows].cpu().numpy(), ri)
        R.within("topk_w", R.host(w[rows]), rw, weight_bound(some, ri, rw, 1.0))
        R.within("dlogits", R.host(d[rows]), ref, 200 * 2.0 ** -24)  # weights below 1, as in check_bwd
    assert not torch.isnan(d).any()


def test_more_tokens_than_one_grid_row():
    """2^28 tokens and some over two experts: more than 2^32 threads."""
    T = (1 << 28) + 1001
    note(f"route T={T} E=2")
    l = torch.zeros(T, 2, device="cuda")
    l[::3, 1] = 2.0
    idx, w = torch.full((T, 1), -1, dtype=torch.int32, device="cuda"), torch.full((T, 1), 7.0, device="cuda")
    moe.moe_route_scored(l, None, idx, w, 1, R.SIGMOID, renormalize=False)
    torch.cuda.synchronize()
    third = torch.arange(T, device="cuda") % 3 == 0
    assert torch.equal(idx[:, 0] == 1, third) and ((idx == 0) | (idx == 1)).all()
    two = 1.0 / (1.0 + np.exp(-2.0))  # the other tokens' score is 1 / 2
    assert (w[third] - two).abs().max() <= 8 * 2.0 ** -24 and (w[~third] - 0.5).abs().max() <= 8 * 2.0 ** -24
    d = torch.full((T, 2), 7.0, device="cuda")
    moe.moe_route_scored_bwd(l, idx, w, d, R.SIGMOID, False)  # the weights as their own gradient
    torch.cuda.synchronize()
    assert (d[third, 1] - two * two * (1 - two)).abs().max() <= 16 * 2.0 ** -24 and (d[third, 0] == 0).all()
    assert (d[~third, 0] - 0.125).abs().max() <= 16 * 2.0 ** -24 and (d[~third, 1] == 0).all()


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
def test_route_near_ties_are_decided_exactly(score):
    """Choice scores closer than fp32 resolves: biases that cancel the scores' differences down to ~1e-9, logits
    one fp32 step apart, and scores next to 1 and next to 0."""
    rng = np.random.default_rng(6)
    T, E, k = 200, 64, 8
    l = np.float32(rng.standard_normal((T, E)))
    base = np.float32(rng.standard_normal(E))
    l[:100] = base  # one row for all: its scores can be cancelled by a bias
    bias = np.float32(0.9 - R.scores(base[None].astype(np.float64), score)[0])
    check(l, bias, k, score)
    check(l, bias, k, score, 8, 3, 2)
    step = np.float32(1.0)
    rows = []
    for _ in range(100):
        v = np.full(E, step, np.float32)
        for j in range(rng.integers(0, 5)):
            up = rng.random(E) < 0.5
            v = np.where(up, np.nextafter(v, np.float32(2)), v)
        rows.append(v)
    check(np.stack(rows), None, k, score)
    check(np.stack(rows), np.zeros(E), k, score)
    check(np.stack(rows), None, k, score, 8, 2, 2)
    wide = np.concatenate([rng.uniform(14, 34, (50, E)), -rng.uniform(20, 90, (50, E)), rng.uniform(40, 90, (20, E))])
    check(wide, None, k, score)
    check(wide, None, k, score, 8, 2, 1, False)
    check(wide[:50], np.zeros(E), k, score)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("E,k,groups", [(16, 4, 4), (128, 8, 8), (37, 5, 1)])
def test_route_unavailable_experts_and_nan(score, E, k, groups):
    rng = np.random.default_rng(7)
    l = rng.standard_normal((60, E))
    l[:20][rng.random((20, E)) < 0.5] = -INF      # half of them
    l[20:30] = -INF                               # a row with nothing left
    l[30:40, :-2] = -INF                          # fewer than k left
    l[30, 1] = 0.3
    l[40:44, 3] = np.nan
    l[44:46, 5] = INF
    l[46, 2:4] = np.nan
    l[47] = np.finfo(np.float32).min              # the lowest finite value
    l[48, ::2] = np.finfo(np.float32).min
    l[49] = np.finfo(np.float32).max
    bias = 0.3 * rng.standard_normal(E)
    other = bias.copy()
    other[1], other[4], other[6] = -INF, INF, np.nan
    for b in (None, bias, other):
        for renorm in (True, False):
            check(l, b, k, score, renorm=renorm)
            if groups > 1:
                check(l, b, k, score, groups, 2, 1, renorm)
                check(l, b, k, score, groups, 2, 2, renorm)


def bwd(l, idx, g, score, renorm, scale):
    T, E = l.shape
    note(f"route bwd T={T} E={E} k={idx.shape[1]} score={score} renorm={renorm}")
    d = torch.full((T, E), 7.0, device="cuda")
    moe.moe_route_scored_bwd(torch.from_numpy(np.float32(l)).cuda(), torch.from_numpy(np.int32(idx)).cuda(),
                             torch.from_numpy(np.float32(g)).cuda(), d, score, renorm, scale)
    torch.cuda.synchronize()
    return R.host(d)


def check_bwd(l, idx, g, score, renorm, scale):
    l, g = (np.asarray(a, np.float32).astype(np.float64) for a in (l, g))
    ref = R.route_bwd(l, idx, g, score, renorm, scale)
    got = bwd(l, idx, g, score, renorm, scale)
    # every term is a product of a probability <= 1, scale and g; differences of such terms, each with the
    # steps of weight_bound and the sum over k
    top = np.where(np.isfinite(l), np.abs(l), 0).max(1, keepdims=True)
    unit = abs(scale) * np.abs(g).max(1, keepdims=True) * (1 if renorm or score == R.SIGMOID else 2)
    R.within("dlogits", got, ref, (8 * (top + 4) + 32 + 2 * l.shape[1]) * 2.0 ** -24 * unit)
    if renorm or score == R.SIGMOID:  # exact zeros elsewhere
        off = np.ones(l.shape, bool)
        np.put_along_axis(off, idx.astype(np.int64), False, axis=1)
        assert not got[off].any()


@pytest.mark.parametrize("T,E,k,groups,top_groups", SHAPES)
@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward(T, E, k, groups, top_groups, score, renorm):
    rng = np.random.default_rng(T + E)
    l = rng.standard_normal((T, E)) * 1.5
    idx, _ = R.route(l, None, k, score)
    check_bwd(l, idx, rng.standard_normal((T, k)), score, renorm, 2.5)
    # any selection, not only the best
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    check_bwd(l, idx, rng.standard_normal((T, k)), score, renorm, -0.5)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_masked_rows_and_repeats(score, renorm):
    rng = np.random.default_rng(9)
    l = rng.standard_normal((24, 20))
    l[:4] = -INF                       # nothing available
    l[4:8, :17] = -INF                 # fewer than k available
    idx, _ = R.route(l, None, 6, score)
    g = rng.standard_normal((24, 6))
    check_bwd(l, idx, g, score, renorm, 1.0)
    idx[10] = [3, 3, 3, 5, 5, 1]       # an index listed twice counts twice
    check_bwd(l, idx, g, score, renorm, 1.0)
    idx[11, 2] = -1                    # outside: left out
    idx[12, 0] = 20
    got = bwd(l, idx, g, score, renorm, 1.0)
    assert np.isfinite(got).all()
    for t, j in ((11, 2), (12, 0)):
        keep = [i for i in range(6) if i != j]
        ref = R.route_bwd(np.float32(l[t:t + 1]).astype(np.float64), idx[t:t + 1, keep],
                          np.float32(g[t:t + 1, keep]).astype(np.float64), score, renorm, 1.0)
        R.within("dlogits without the index", got[t:t + 1], ref, 200 * 2.0 ** -24 * np.abs(g[t]).max() * 2)


def test_one_renormalised_weight_has_no_gradient():
    rng = np.random.default_rng(10)
    l = rng.standard_normal((50, 32))
    idx = np.argsort(-l, axis=1)[:, :1].astype(np.int32)
    for score in (R.SOFTMAX, R.SIGMOID):
        assert not bwd(l, idx, rng.standard_normal((50, 1)), score, True, 2.0).any()


@pytest.mark.parametrize("T,H,E,dtype", [(64, 128, 8, "f32"), (300, 384, 128, "bf16"), (33, 104, 20, "bf16")])
def test_router_products_of_given_dlogits(T, H, E, dtype):
    """The same products as moe_router_bwd makes of its own dlogits, bit for bit, and the formula's."""
    note(f"router products T={T} H={H} E={E} {dtype}")
    rng = np.random.default_rng(12)
    x, wr = R.rounded(rng.standard_normal((T, H)), dtype), R.rounded(0.05 * rng.standard_normal((H, E)), dtype)
    dl = np.float32(rng.standard_normal((T, E)))
    xd, wd, dld = R.dev(x, dtype), R.dev(wr, dtype), torch.from_numpy(dl).cuda()
    dw, dx0 = torch.empty_like(wd), R.dev(rng.standard_normal((T, H)), dtype)
    ws = torch.empty(max(16, moe.moe_router_workspace_bytes(T, H, E)), dtype=torch.uint8, device="cuda")
    for accumulate in (False, True):
        dx = dx0.clone()
        moe.moe_router_bwd_dlogits(xd, wd, dld, dw, dx, accumulate, ws)
        torch.cuda.synchronize()
        ref = dl.astype(np.float64) @ wr.T + (R.host(dx0) if accumulate else 0)
        # bf16 layers multiply dlogits as two bf16 parts: 2^-16 of each term
        part = 2.0 ** -16 if dtype == "bf16" else 0.0
        size = np.abs(dl).astype(np.float64) @ np.abs(wr).T
        R.within("dx", R.host(dx), ref, R.U[dtype] * np.abs(ref) + (part + (E + 4) * 2.0 ** -23) * size
                 + 2.0 ** -23 * np.abs(ref))
        ref = x.T @ dl.astype(np.float64)
        size = np.abs(x).T @ np.abs(dl).astype(np.float64)
        R.within("dw_r", R.host(dw), ref, R.U[dtype] * np.abs(ref) * 1.01 + (part + (T + 4) * 2.0 ** -23) * size)
    idx, w = R.route(np.float32(rng.standard_normal((T, E))), None, 2, R.SOFTMAX)
    g = torch.from_numpy(np.float32(rng.standard_normal((T, 2)))).cuda()
    wt = torch.from_numpy(np.float32(w)).cuda()
    own, dx1, dw1 = torch.empty(T, E, device="cuda"), dx0.clone(), torch.empty_like(wd)
    moe.moe_router_bwd(xd, wd, torch.from_numpy(idx).cuda(), wt, g, own, dw1, dx1, True, ws)
    dx2 = dx0.clone()
    moe.moe_router_bwd_dlogits(xd, wd, own, dw, dx2, True, ws)
    torch.cuda.synchronize()
    assert torch.equal(dx1, dx2) and torch.equal(dw, dw1)
