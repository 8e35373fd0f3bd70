"""The balance loss over ragged batches of many sequences: however rows lie over the
sequences, every run of rows is summed once, long sequences keep their precision, and
repeats give the same bits."""
import numpy as np
import pytest
import torch

import step_ref as S
from expert_grouped_gemm_top_amd import moe
from moe_cases import note
from test_gpu_balance import case, check, forward, gpu

pytestmark = pytest.mark.gpu


def cuts(kind, n_seq, T, seed):
    rng = np.random.default_rng(seed)
    if kind == "one long":  # nearly all rows in one sequence
        at = n_seq // 3
        return [0] + [2 * i for i in range(1, at + 1)] + [T - 2 * (n_seq - 1 - at) + 2 * i for i in range(n_seq - at)]
    if kind == "blocks":  # borders on, before and behind multiples of the runs' 64 rows
        return sorted(np.clip(64 * rng.integers(0, T // 64 + 1, n_seq + 1) + rng.integers(-1, 2, n_seq + 1), 0, T).tolist())
    if kind == "late":  # rows in front of the first sequence and behind the last, many empty ones
        return sorted(rng.integers(T // 3, T // 2, n_seq + 1).tolist())
    return [-3] * (n_seq // 2) + sorted(rng.integers(-3, T + 4, n_seq + 1 - n_seq // 2).tolist())  # empty ones first, cut off


@pytest.mark.parametrize("kind", ["one long", "blocks", "late", "empty"])
@pytest.mark.parametrize("n_seq,T", [(2, 300), (63, 4000), (64, 4000), (65, 4000), (66, 70001), (130, 1000), (600, 5000),
                                     (4097, 9000)])
def test_ragged(kind, n_seq, T):
    off = cuts(kind, n_seq, T, n_seq)
    assert len(off) == n_seq + 1 and (np.diff(off) >= 0).all()
    l, idx = case(T, 20, 2, n_seq + T)
    check(l, idx, off, n_seq % 2)


def test_many_empty_sequences():
    """65535 sequences, of which three have rows."""
    T, E, n = 1000, 12, 65535
    off = np.zeros(n + 1, np.int32)
    off[100:] = 70
    off[40000:] = 640
    off[65535:] = 990
    l, idx = case(T, E, 3, 9)
    counts, mean, loss = (t.cpu().numpy() for t in forward(l, idx, off.tolist(), 0, 1.0))
    rows = [99, 39999, 65534]
    c, m, want = S.balance(l, idx, [0, 70, 640, 990], 0, 1.0)
    assert np.array_equal(counts[rows], c) and not counts[np.delete(np.arange(n), rows)].any()
    assert (np.abs(mean[rows] - m) <= 1e-5 * m).all() and not mean[np.delete(np.arange(n), rows)].any()
    assert abs(loss[0] - want) <= 1e-5 * want


@pytest.mark.parametrize("score", [0, 1])
def test_a_long_sequence_among_many_keeps_its_precision(score):
    """500000 equal rows, nearly all in one of 1000 sequences: shares of 1 / 200.  A share is off by 40 roundings (its
    exponential, 13 a lane and four additions, the reciprocal), a run's sum by 16 rows a thread, two and sixteen more."""
    T, E, n = 500000, 200, 1000
    off = cuts("one long", n, T, 0)
    note("balance, one long sequence")
    logits = torch.zeros(T, E, device="cuda")
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    counts, mean, loss = forward(np.empty((T, E), np.float32), np.zeros((T, 1), np.int32), off, score, 1.0, logits=logits)
    sizes = torch.from_numpy(np.diff(off)).cuda()
    assert torch.equal(counts[:, 0].long(), sizes) and not counts[:, 1:].any()
    assert float((mean.double() * E - 1).abs().max()) <= (40 + 34) * 2.0 ** -23
    assert abs(float(loss) - 1.0) <= (40 + 34 + 2) * 2.0 ** -23
    again = forward(np.empty((T, E), np.float32), idx.cpu().numpy(), off, score, 1.0, logits=logits)
    assert torch.equal(again[1], mean) and torch.equal(again[2], loss)


def test_replays_with_other_offsets():
    """A captured call takes the offsets that are there when it is replayed."""
    T, E, n = 3000, 64, 90
    l, idx = case(T, E, 4, 3)
    logits, index = gpu(l, torch.float32), gpu(idx, torch.int32)
    off = gpu(cuts("blocks", n, T, 1), torch.int32)
    ws = torch.empty(moe.moe_balance_loss_workspace_bytes(T, E, n), dtype=torch.uint8, device="cuda")
    new = lambda: (torch.empty(n, E, dtype=torch.int32, device="cuda"), torch.empty(n, E, device="cuda"), torch.empty(1, device="cuda"))  # noqa: E731
    out = new()
    moe.moe_balance_loss_fwd(logits, index, *out, ws, seq_offsets=off)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_balance_loss_fwd(logits, index, *out, ws, seq_offsets=off)
    for i, kind in enumerate(("one long", "late", "empty", "blocks")):
        at = cuts(kind, n, T, 10 + i)
        off.copy_(gpu(at, torch.int32))
        g.replay()
        ref = forward(l, idx, at, 0, 1.0)
        for a, b in zip(out, ref):
            assert torch.equal(a, b), kind
