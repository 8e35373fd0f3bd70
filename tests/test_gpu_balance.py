"""The balance loss, its counts and its gradient against the 64-bit formula: sizes
around the kernels' borders, ragged and empty sequences, padding, unavailable
experts, confident tokens, and the ways a caller may run it."""
import numpy as np
import pytest
import torch

import step_ref as S
from block_ref import U, host, within
from expert_grouped_gemm_top_amd import moe
from moe_cases import note

pytestmark = pytest.mark.gpu


def case(T, E, k, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    l = (spread * rng.standard_normal((T, E)) + 0.5 * rng.standard_normal(E)).astype(np.float32)
    idx = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    return l, idx


def gpu(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda()


def forward(l, idx, offsets, score, alpha, logits=None, stream=None):
    T, E = l.shape
    n = 1 if offsets is None else len(offsets) - 1
    out = (torch.full((n, E), 7, dtype=torch.int32, device="cuda"), torch.full((n, E), 7.0, device="cuda"),
           torch.full((1,), 7.0, device="cuda"))
    need = moe.moe_balance_loss_workspace_bytes(T, E, n)
    ws = torch.full((max(need, 16),), 0xff, dtype=torch.uint8, device="cuda")
    moe.moe_balance_loss_fwd(gpu(l, torch.float32) if logits is None else logits, gpu(idx, torch.int32), *out, ws, score=score,
                             alpha=alpha, seq_offsets=None if offsets is None else gpu(offsets, torch.int32), stream=stream)
    torch.cuda.synchronize()
    return out


# A share's relative error: exp and its argument's rounding, (span + 4) 2^-23, and as much again for the sum and its
# reciprocal with 24 additions of positive terms; a sigmoid's logits enter twice.
def share_error(l):
    fine = np.abs(l[np.isfinite(l)])
    return (4 * (fine.max() if fine.size else 0.0) + 60) * 2.0 ** -23


def check(l, idx, offsets, score, alpha=0.01, k=None, dloss=None, add=None):
    T, E = l.shape
    off = [0, T] if offsets is None else offsets
    note(f"balance T={T} E={E} k={idx.shape[1]} score={score} offsets={off[:6]}")
    counts, mean, loss = forward(l, idx, offsets, score, alpha)
    rc, rm, rl = S.balance(l, idx, off, score, alpha)
    assert np.array_equal(counts.cpu().numpy(), rc)
    err = share_error(l) + (110 + T / 64) * 2.0 ** -23  # and the additions over the rows
    within("mean_p", host(mean), rm, err * np.abs(np.nan_to_num(rm)) + 1e-37)
    within("loss", host(loss), np.array([rl]), 2 * err * abs(np.nan_to_num(rl)) + 1e-37)
    d = torch.full((T, E), 7.0, device="cuda")
    kw = dict(score=score, alpha=alpha, seq_offsets=None if offsets is None else gpu(offsets, torch.int32),
              dloss=None if dloss is None else torch.tensor([dloss], device="cuda"))
    logits = gpu(l, torch.float32)
    moe.moe_balance_loss_bwd(logits, counts, d, idx.shape[1], **kw)
    ref, size = S.balance_bwd(l, rc, idx.shape[1], off, score, alpha, 1.0 if dloss is None else np.float64(np.float32(dloss)))
    bound = 3 * share_error(l) * np.nan_to_num(size) + 1e-37
    within("dlogits", host(d), ref, bound)
    a = np.random.default_rng(5).standard_normal((T, E)).astype(np.float32)
    d2 = torch.full((T, E), 7.0, device="cuda")
    moe.moe_balance_loss_bwd(logits, counts, d2, idx.shape[1], dl_add=gpu(a, torch.float32), **kw)
    within("dlogits + dl_add", host(d2), ref + a, bound + U["f32"] * np.abs(np.nan_to_num(ref + a)))
    d3 = gpu(a, torch.float32)
    moe.moe_balance_loss_bwd(logits, counts, d3, idx.shape[1], dl_add=d3, **kw)
    torch.cuda.synchronize()
    assert torch.equal(d3.view(torch.int32), d2.view(torch.int32))
    return d


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 1), (2, 16, 16), (63, 7, 3), (64, 60, 4), (65, 128, 8), (256, 256, 8),
                                   (257, 255, 5), (1030, 128, 8), (4099, 33, 2), (16384, 256, 8), (70001, 20, 1)])
def test_sizes(T, E, k, score):
    l, idx = case(T, E, k, T + E)
    check(l, idx, None, score, dloss=0.3 if T % 2 else None)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,offsets", [(300, 64, [0, 1, 1, 130, 300]), (300, 64, [0, 0]), (300, 30, [10, 20]),
                                         (257, 128, [0, 0, 0, 257]), (500, 128, [7, 200, 200, 201, 450]),
                                         (5, 8, [0, 1, 2, 3, 4, 5]), (2000, 256, list(range(0, 1801, 3))),
                                         (64, 16, [-5, 30, 1 << 30])])
def test_sequences(T, E, offsets, score):
    l, idx = case(T, E, 4, T)
    d = check(l, idx, offsets, score)
    outside = S.sequences(T, offsets) < 0
    assert (host(d)[outside] == 0).all()


@pytest.mark.parametrize("score", [0, 1])
def test_unavailable_experts_and_confident_tokens(score):
    l, idx = case(200, 64, 4, 1)
    l[3, 5:] = -np.inf  # a few left
    l[4] = -np.inf      # none left
    l[5] = -200.0 - np.arange(64)  # every sigmoid underflows
    l[6, 7] = 60.0      # all but one share vanish
    l[7, 9] = 25.0
    l[:, 11] = -np.inf  # an expert that no token may take
    check(l, idx, None, score)


@pytest.mark.parametrize("score", [0, 1])
def test_nan_stays_in_its_sequence(score):
    l, idx = case(90, 32, 2, 2)
    l[40, 3] = np.nan
    offsets = [0, 30, 60, 80]
    l[85] = np.nan  # behind the last sequence: nothing
    counts, mean, loss = forward(l, idx, offsets, score, 1.0)
    m = host(mean)
    assert np.isfinite(m[[0, 2]]).all() and np.isnan(m[1]).all() and np.isnan(host(loss)).all()
    d = torch.zeros(90, 32, device="cuda")
    moe.moe_balance_loss_bwd(gpu(l, torch.float32), counts, d, 2, score=score, seq_offsets=gpu(offsets, torch.int32))
    h = host(d)
    assert np.isnan(h[40]).all() and np.isfinite(np.delete(h, 40, 0)).all()


def test_indexes_outside_and_twice():
    l, idx = case(100, 16, 3, 3)
    idx[0] = [-1, 16, 2**31 - 1]
    idx[1] = [4, 4, 4]
    check(l, idx, None, 0)


def test_a_difference_quotient():
    """The gradient is that of the forward with the counts held fixed."""
    l, idx = case(40, 12, 2, 4)
    offsets = [0, 15, 33]
    for score in (0, 1):
        counts, _, _ = forward(l, idx, offsets, score, 1.0)
        d = torch.empty(40, 12, device="cuda")
        moe.moe_balance_loss_bwd(gpu(l, torch.float32), counts, d, 2, score=score, seq_offsets=gpu(offsets, torch.int32))
        c, h = counts.cpu().numpy(), 1e-4
        for t, e in ((0, 3), (14, 0), (15, 7), (32, 11), (33, 2)):
            f = []
            for sign in (1, -1):
                moved = l.astype(np.float64)
                moved[t, e] += sign * h
                p, seq = S.shares(moved, score), S.sequences(40, offsets)
                f.append(12 / 2 / 33 * sum((c[s] * p[seq == s].mean(0)).sum() for s in range(2)))
            assert abs((f[0] - f[1]) / (2 * h) - float(d[t, e])) <= 1e-6 * np.abs(host(d)).max() + 1e-7


def test_unaligned_rows_and_other_streams():
    l, idx = case(333, 64, 4, 6)
    flat = torch.empty(333 * 64 + 1, device="cuda")
    flat[1:] = gpu(l, torch.float32).view(-1)
    ref = forward(l, idx, None, 1, 0.5)
    got = forward(l, idx, None, 1, 0.5, logits=flat[1:].view(333, 64))
    for a, b in zip(ref, got):
        assert torch.allclose(a.double(), b.double(), rtol=2.0 ** -20, atol=0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for a, b in zip(ref, forward(l, idx, None, 1, 0.5, stream=s)):
        assert torch.equal(a, b)


def test_captured_replays():
    """Replays with new logits, eager work between them, one workspace for two graphs."""
    T, E, k, offsets = 3000, 128, 8, [0, 900, 900, 2500]
    l, idx = case(T, E, k, 7)
    logits, index, off = gpu(l, torch.float32), gpu(idx, torch.int32), gpu(offsets, torch.int32)
    ws = torch.empty(moe.moe_balance_loss_workspace_bytes(T, E, 3), dtype=torch.uint8, device="cuda")

    def buffers():
        return (torch.empty(3, E, dtype=torch.int32, device="cuda"), torch.empty(3, E, device="cuda"),
                torch.empty(1, device="cuda"), torch.empty(T, E, device="cuda"))

    def step(b):
        moe.moe_balance_loss_fwd(logits, index, *b[:3], ws, score=1, seq_offsets=off)
        moe.moe_balance_loss_bwd(logits, b[0], b[3], k, score=1, seq_offsets=off)

    sets = [buffers(), buffers()]
    eager = buffers()
    step(eager)
    graphs = []
    for b in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(b)
        graphs.append(g)
    for i in range(4):
        logits.copy_(gpu(case(T, E, k, 20 + i)[0], torch.float32))
        for b in sets:
            for x in b:
                x.fill_(3)
        step(eager)
        graphs[i % 2].replay()
        graphs[1 - i % 2].replay()
        torch.cuda.synchronize()
        for b in sets:
            for x, y in zip(b, eager):
                assert torch.equal(x, y)


def test_logits_past_32_bit_offsets():
    """2.1e9 logits in two sequences, all equal but in the last row: its share and its gradient."""
    T, E = (1 << 23) + 5, 256
    l = torch.zeros(T, E, device="cuda")
    l[T - 1, E - 1] = 8
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    idx[T - 3:] = E - 1
    off = torch.tensor([0, T - 3, T], dtype=torch.int32, device="cuda")
    counts, mean = torch.zeros(2, E, dtype=torch.int32, device="cuda"), torch.zeros(2, E, device="cuda")
    loss = torch.zeros(1, device="cuda")
    ws = torch.empty(moe.moe_balance_loss_workspace_bytes(T, E, 2), dtype=torch.uint8, device="cuda")
    moe.moe_balance_loss_fwd(l, idx, counts, mean, loss, ws, seq_offsets=off)
    d = torch.full((T, E), 7.0, device="cuda")
    moe.moe_balance_loss_bwd(l, counts, d, 1, seq_offsets=off)
    torch.cuda.synchronize()
    assert counts[0, 0] == T - 3 and counts[1, E - 1] == 3 and int(counts.sum()) == T
    assert (mean[0].double() - 1 / E).abs().max() <= 200 * 2.0 ** -23 / E + (T / 1024 / 64) * 2.0 ** -24 / E
    top = np.exp(8.0) / (np.exp(8.0) + E - 1)
    want = E / T * ((T - 3) / E + 3 * (2 / E + top) / 3)
    assert abs(float(loss) - want) <= 1e-3 * want
    f = E / T / 3  # of the last sequence's rows
    assert abs(float(d[T - 1, E - 1]) - f * top * 3 * (1 - top)) <= 1e-5 * f * top * 3 * (1 - top)
    assert abs(float(d[T - 2, 0]) + f / E * 3 / E) <= 1e-5 * f / E * 3 / E
    first = E / T / (T - 3) / E * (T - 3) * (1 - 1 / E)
    assert abs(float(d[0, 0]) - first) <= 1e-5 * first and abs(float(d[T - 4, 0]) - first) <= 1e-5 * first
    del l, d
    torch.cuda.empty_cache()


def test_launches():
    for T, n in ((256, 1), (257, 2)):
        l, idx = case(T, 16, 2, 8)
        before = moe.moe_launch_count()
        forward(l, idx, None, 0, 1.0)
        assert moe.moe_launch_count() - before == n
