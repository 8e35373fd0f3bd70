"""Cross entropy over a vocabulary without kept logits, and its gradients, against
the 64-bit formula: sizes around the tiles and pieces, tokens that are not counted
(whatever lies in their rows), padding columns, confident tokens, and the ways a
caller may run it."""
import numpy as np
import pytest
import torch

import step_ref as S
from block_ref import DT, U, dev, host, rounded, within
from expert_grouped_gemm_top_amd import moe
from moe_cases import note

pytestmark = pytest.mark.gpu


def case(T, H, V, dtype, seed, vocab=None, ignored=0.3, spread=2.0):
    rng = np.random.default_rng(seed)
    vocab = V if vocab is None else vocab
    x = rng.standard_normal((T, H))
    w = spread * H ** -0.5 * rng.standard_normal((H, V))
    y = rng.integers(0, vocab, T)
    x += (8 * rng.random((T, 1))) * w[:, y].T / (w[:, y] ** 2).sum(0)[:, None]
    y[rng.random(T) < ignored] = -100
    return rounded(x, dtype), rounded(w, dtype), y.astype(np.int32), vocab


class Buffers:
    def __init__(self, T, H, V, dtype, dx=True, dw=True):
        d = DT[dtype]
        full = lambda *s, dt=torch.float32: torch.full(s, 7, dtype=dt, device="cuda")  # noqa: E731
        self.loss, self.lse, self.mean = full(T), full(T), full(2)
        self.dx, self.dw = full(T, H, dt=d) if dx else None, full(H, V, dt=d) if dw else None
        self.ws = full(moe.moe_vocab_loss_workspace_bytes(T, H, V, d), dt=torch.uint8)
        self.ws.fill_(0xff)  # NaN wherever it is read unwritten

    def step(self, x, w, y, vocab, dloss=None, scale=1.0, stream=None):
        moe.moe_vocab_loss_fwd(x, w, y, self.loss, self.lse, self.mean, self.ws, vocab=vocab, stream=stream)
        if self.dx is not None or self.dw is not None:
            moe.moe_vocab_loss_bwd(x, w, y, self.loss, self.lse, self.mean, self.dx, self.dw, self.ws, dloss, scale, vocab, stream)

    def outputs(self):
        return [t for t in (self.loss, self.lse, self.mean, self.dx, self.dw) if t is not None]


# A logit of H terms is off by H 2^-23 of their sizes; a statistic by twice that, its own
# exponentials' and logarithms' roundings (|logit| + 64) 2^-23 and the additions' V 2^-24.
def check(T, H, V, dtype, seed=0, vocab=None, ignored=0.3, weighted=False, scale=1.0, dx=True, dw=True, spoil=False):
    note(f"vocab T={T} H={H} V={V} {dtype} vocab={vocab} ignored={ignored} weighted={weighted} dx={dx} dw={dw}")
    x, w, y, vocab = case(T, H, V, dtype, seed, vocab, ignored)
    dl = np.random.default_rng(seed + 1).random(T).astype(np.float32).astype(np.float64) if weighted else None
    ref = S.vocab(x, w, y, vocab, dl, scale)
    if spoil:
        x = x.copy()
        x[y < 0] = np.nan
        x[np.flatnonzero(y < 0)[::2]] = np.inf
    b = Buffers(T, H, V, dtype, dx, dw)
    b.step(dev(x, dtype), dev(w, dtype), torch.from_numpy(y).cuda(), vocab, None if dl is None else torch.from_numpy(dl).float().cuda(), scale)
    torch.cuda.synchronize()
    off = 2 * H * 2.0 ** -23 * ref["size"] + (np.abs(ref["lse"]) + ref["size"] + 64) * 2.0 ** -23 + V * 2.0 ** -24
    within("lse", host(b.lse), ref["lse"], off + U["f32"] * np.abs(ref["lse"]))
    within("loss", host(b.loss), ref["loss"], off + U["f32"] * np.abs(ref["loss"]))
    within("mean", host(b.mean), ref["mean"], np.array([off.max(), 0]) + 2 * U["f32"] * np.abs(ref["mean"]))
    # A term of dx is f (q - [v = y]) w, with q - [v = y] rounded to the type: U of it.  One of dw is (f x) (q - [v = y])
    # with both factors rounded: (1 + U)^2 - 1 = 2 U + U^2.  Either sum is rounded once more as it is stored.
    rel = 2 * off.max() + 16 * 2.0 ** -23  # of f and q
    for name, got, want, size, terms, rounded_factors in (("dx", b.dx, ref["dx"], ref["sx"], vocab, U[dtype]),
                                                          ("dw", b.dw, ref["dw"], ref["sw"], ref["n"], 2 * U[dtype] + U[dtype] ** 2)):
        if got is not None:
            within(name, host(got), want, (rel + rounded_factors + terms * 2.0 ** -23) * size + U[dtype] * np.abs(want) + 1e-38)
    assert (host(b.loss)[(y < 0) | (y >= vocab)] == 0).all() and (host(b.lse)[(y < 0) | (y >= vocab)] == 0).all()
    if dw:
        assert (host(b.dw)[:, vocab:] == 0).all()
    return b


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,V,vocab", [(1, 8, 8, 1), (1, 64, 40, 37), (2, 128, 256, None), (7, 200, 264, 258), (31, 72, 1008, 1003),
                                         (33, 64, 2048, None), (64, 512, 776, 770), (127, 136, 1032, None), (129, 256, 1280, 1025),
                                         (333, 200, 1008, 1003), (300, 1024, 520, None)])
def test_sizes(T, H, V, vocab, dtype):
    check(T, H, V, dtype, seed=T, vocab=vocab, weighted=T % 2 == 0, scale=0.5 if T > 100 else 1.0)


@pytest.mark.parametrize("T,H,V,vocab", [(1030, 512, 4104, 4099), (4099, 256, 2056, None), (257, 2048, 8192, None), (16, 2048, 32000, None)])
def test_larger_bf16(T, H, V, vocab):
    check(T, H, V, "bf16", seed=T, vocab=vocab, weighted=True)


@pytest.mark.parametrize("ignored", [0.3, 0.99])
def test_several_pieces(ignored):
    """Vocabularies of more than one piece, the last of odd width."""
    T = 20000
    x, w, y, vocab = case(T, 64, 9000, "bf16", 3, 8997, ignored)
    b = Buffers(T, 64, 9000, "bf16")
    d = [dev(x, "bf16"), dev(w, "bf16"), torch.from_numpy(y).cuda()]
    before = moe.moe_launch_count()
    b.step(*d, vocab)
    torch.cuda.synchronize()
    assert moe.moe_launch_count() - before > 3 + 3 + 2  # more than one piece
    X, W = d[0].double(), d[1][:, :vocab].double()
    keep = d[2] >= 0
    l = X @ W
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    p[torch.arange(T, device="cuda"), d[2].long().clamp(min=0)] -= 1
    p *= (keep.double() / keep.sum())[:, None]
    off = 1e-4  # the losses' bound at these sizes: logits of 64 terms below 60 in size
    assert ((b.lse.double() - lse) * keep).abs().max() <= off
    for got, want, size, factors in ((b.dx, p @ W.t().contiguous(), p.abs() @ W.abs().t().contiguous(), 1),
                                     (b.dw[:, :vocab], X.t().contiguous() @ p, X.abs().t().contiguous() @ p.abs(), 2.01)):
        bound = (2 * off + factors * U["bf16"] + T * 2.0 ** -23) * size + U["bf16"] * want.abs()  # as in check()
        assert ((got.double() - want).abs() <= bound).all()
    assert (b.dw[:, vocab:] == 0).all() and (b.dx[~keep] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dx,dw", [(True, False), (False, True), (False, False)])
def test_either_gradient_alone(dx, dw, dtype):
    a, b = check(200, 128, 1024, dtype, seed=4, dx=dx, dw=dw), check(200, 128, 1024, dtype, seed=4)
    if dw:
        assert torch.equal(a.dw, b.dw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ignored", [0.0, 0.5, 0.97, 1.0])
def test_rows_that_are_not_counted_may_hold_anything(ignored, dtype):
    check(150, 96, 520, dtype, seed=5, vocab=515, ignored=ignored, spoil=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,V,ignored", [(2100, 264, 2056, 0.6), (2100, 264, 2056, 0.97), (1700, 136, 4104, 0.9),
                                           (1025, 72, 1000, 1.0), (1030, 512, 24, 0.8), (900, 128, 3000, 0.95)])
def test_few_of_many_tokens_are_counted(T, H, V, ignored, dtype):
    """The slices of dx are cut again where most tokens are not counted."""
    check(T, H, V, dtype, seed=T, vocab=V - 3, ignored=ignored, weighted=True, spoil=True)


def test_targets_outside_are_not_counted():
    x, w, y, _ = case(64, 64, 104, "bf16", 6, 100, 0.0)
    y[:6] = [-1, 100, 103, 104, 2**31 - 1, -2**31]
    ref = S.vocab(x, w, y, 100)
    b = Buffers(64, 64, 104, "bf16")
    b.step(dev(x, "bf16"), dev(w, "bf16"), torch.from_numpy(y).cuda(), 100)
    assert ref["n"] == 58 and (host(b.loss)[:6] == 0).all() and (host(b.dx)[:6] == 0).all()
    assert float(b.mean[1]) == np.float32(1 / 58)


def test_confident_tokens_keep_their_digits():
    """Losses down to 1e-8 and the gradients that go with them, which a difference of rounded numbers would lose.  All
    logits are whole, so that nothing else is rounded."""
    H = V = 64
    x = np.zeros((8, H))
    w = np.eye(H)
    for t in range(8):
        x[t, t] = 4.0 * t
    y = np.arange(8, dtype=np.int32)
    ref = S.vocab(x, w, y, V)
    b = Buffers(8, H, V, "f32")
    b.step(dev(x, "f32"), dev(w, "f32"), torch.from_numpy(y).cuda(), V)
    assert (np.abs(host(b.loss) - ref["loss"]) <= 200 * 2.0 ** -24 * ref["loss"]).all() and ref["loss"].min() < 1e-10
    diag = np.arange(8)
    assert (np.abs(host(b.dx)[diag, diag] - ref["dx"][diag, diag]) <= 300 * 2.0 ** -24 * np.abs(ref["dx"][diag, diag])).all()


@pytest.mark.parametrize("far", [2.0 ** 20, 2.0 ** 40, float("inf")])
def test_a_target_far_below_leaves_the_others_their_digits(far):
    """lse and the others' gradients do not pass through the target's logit.  All logits are whole: lse is off by the
    exponentials' and the logarithm's roundings, below 64 2^-24, a gradient by that, its own and its product's."""
    H = V = 16
    x, w = np.zeros((3, H)), np.eye(H)
    x[0, :4], x[1, 5:9], x[2, 3] = [1, 2, 3, 4], [7, 0, 7, 1], 2
    y = np.array([15, 14, 13], np.int32)
    if np.isfinite(far):
        x[np.arange(3), y] = -far
    else:  # W alone reaches it: an infinite x would make every logit NaN
        x[:, H - 1] = 1
        w[H - 1] = 0
        w[H - 1, 13:] = -far
        y[:] = 15
    with np.errstate(invalid="ignore"):
        l = np.where(np.isinf(w[H - 1])[None, :] & (x[:, H - 1:] != 0), -np.inf, x @ np.where(np.isinf(w), 0, w))
    others = np.where(np.arange(V)[None, :] == y[:, None], -np.inf, l)
    top = others.max(1, keepdims=True)
    lse = (top + np.log(np.exp(others - top).sum(1, keepdims=True)))[:, 0]
    b = Buffers(3, H, V, "f32")
    b.step(dev(x, "f32"), dev(w, "f32"), torch.from_numpy(y).cuda(), V, torch.ones(3, device="cuda"))
    torch.cuda.synchronize()
    within("lse", host(b.lse), lse, 64 * 2.0 ** -24 + np.abs(lse) * 2.0 ** -23)
    if np.isfinite(far):
        own = l[np.arange(3), y]
        within("loss", host(b.loss), lse - own, 64 * 2.0 ** -24 + np.abs(lse - own) * 2.0 ** -23)
        q = np.exp(others - lse[:, None])
        q[np.arange(3), y] = -1
        within("dx", host(b.dx), q @ w.T, 300 * 2.0 ** -24 * (np.abs(q) @ np.abs(w).T))
    else:
        assert (host(b.loss) == np.inf).all()
        q = np.exp(others - lse[:, None])
        q[np.arange(3), y] = -1
        within("dw", host(b.dw), x.T @ q, 300 * 2.0 ** -24 * (np.abs(x).T @ np.abs(q)))


def test_more_tokens_than_the_list_kernels_first_rounds():
    """Two million tokens: their list, 1024 a workgroup, and the products' rows behind it."""
    T, H, V = (1 << 21) + 5, 8, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, device="cuda", generator=g)
    w = torch.randn(H, V, device="cuda", generator=g)
    y = torch.randint(-8, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    b = Buffers(T, H, V, "f32")
    b.step(x, w, y, V)
    keep, rows = y >= 0, torch.arange(T, device="cuda")
    l = (x.double()[:, :, None] * w.double()[None]).sum(1)
    lse = torch.logsumexp(l, 1)
    loss = (lse - l[rows, y.long().clamp(min=0)]) * keep
    assert ((b.lse.double() - lse) * keep).abs().max() <= 64 * 2.0 ** -23 * l.abs().max()
    assert (b.loss.double() - loss).abs().max() <= 64 * 2.0 ** -23 * l.abs().max()
    n = int(keep.sum())
    assert float(b.mean[1]) == np.float32(1 / n) and abs(float(b.mean[0]) - float(loss.sum()) / n) <= 1e-5
    p = torch.exp(l - lse[:, None])
    p[rows, y.long().clamp(min=0)] -= 1
    p *= keep[:, None] / n
    dx = (p[:, None, :] * w.double()[None]).sum(2)
    assert (b.dx.double() - dx).abs().max() <= 200 * 2.0 ** -23 * float((p.abs()[:, None, :] * w.double().abs()[None]).sum(2).max())
    # sums of n terms in fp32, 32 to 64 k at a time in a matrix core's chain: n 2^-24 of their sizes at the most
    dw, size = (x.double()[:, :, None] * p[:, None, :]).sum(0), (x.double().abs()[:, :, None] * p.abs()[:, None, :]).sum(0)
    assert ((b.dw.double() - dw).abs() <= n * 2.0 ** -24 * size).all()


def test_weights_past_32_bit_offsets():
    """4.3e9 weights: their last columns and rows, with classes on both sides of 2^31 and 2^32 elements."""
    T, H, V = 5, 4104, 1 << 20
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(H, V, dtype=torch.bfloat16, device="cuda")
    y = torch.tensor([0, V - 1, V // 2, -1, V - 2], dtype=torch.int32, device="cuda")
    x[:, H - 1] = torch.tensor([1.0, 2.0, -1.0, float("nan"), 0.5])
    x[:, 3] = 1
    w[H - 1, V - 1], w[H - 1, 0], w[3, V // 2], w[H - 1, V - 2] = 8, 4, 6, -3
    b = Buffers(T, H, V, "bf16")
    b.step(x, w, y, V)
    torch.cuda.synchronize()
    # the logits of all but four columns are 0
    at = [0, V // 2, V - 2, V - 1]
    X, W = x[[0, 1, 2, 4]].double().cpu(), w[:, at].double().cpu()
    l = X[:, [3, H - 1]] @ W[[3, H - 1]]
    lse = torch.log(torch.exp(l).sum(1) + (V - 4))
    own = l[torch.arange(4), torch.tensor([0, 3, 1, 2])]
    got = b.loss.double().cpu()[[0, 1, 2, 4]]
    assert (got - (lse - own)).abs().max() <= 1e-4 and float(b.loss[3]) == 0  # a sum of 2^20 terms, and 64 2^-23 of 24
    p = torch.exp(l - lse[:, None])
    p[torch.arange(4), torch.tensor([0, 3, 1, 2])] -= 1
    p /= 4
    dw = X[:, [3, H - 1]].T @ p
    got = b.dw[[3, H - 1]][:, at].double().cpu()
    size = X[:, [3, H - 1]].abs().T @ p.abs()
    assert ((got - dw).abs() <= (3.01 * U["bf16"] + 2e-4) * size).all()  # both factors and the result rounded
    dx = p @ W[[3, H - 1]].T
    got = b.dx[[0, 1, 2, 4]][:, [3, H - 1]].double().cpu()
    assert ((got - dx).abs() <= (2.01 * U["bf16"] + 2e-4) * (p.abs() @ W[[3, H - 1]].T.abs())).all()
    assert (b.dx[3] == 0).all() and int((b.dx != 0).sum()) <= 8
    assert int((b.dw[4:H - 1] != 0).sum()) == 0 and int((b.dw[:3] != 0).sum()) == 0
    del b, w
    torch.cuda.empty_cache()


def test_a_difference_quotient():
    x, w, y, vocab = case(12, 16, 40, "f32", 7, 37)
    b = Buffers(12, 16, 40, "f32")
    b.step(dev(x, "f32"), dev(w, "f32"), torch.from_numpy(y).cuda(), vocab)
    for a, g, at in ((x, b.dx, (0, 3)), (x, b.dx, (5, 15)), (w, b.dw, (2, 36)), (w, b.dw, (15, int(max(y))))):
        f = []
        for h in (1e-5, -1e-5):
            keep = a[at]
            a[at] = keep + h
            f.append(S.vocab(x, w, y, vocab)["mean"][0])
            a[at] = keep
        assert abs((f[0] - f[1]) / 2e-5 - float(g[at])) <= 1e-6


def make(T=700, H=256, V=3000, seed=8):
    x, w, y, vocab = case(T, H, V, "bf16", seed, 2993)
    return [dev(x, "bf16"), dev(w, "bf16"), torch.from_numpy(y).cuda()], vocab


def test_repeated_and_on_other_streams():
    (x, w, y), vocab = make()
    ref, got = Buffers(700, 256, 3000, "bf16"), Buffers(700, 256, 3000, "bf16")
    ref.step(x, w, y, vocab)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    other = Buffers(700, 256, 3000, "bf16")
    for _ in range(3):
        for b, s in zip((got, other), streams):
            b.step(x, w, y, vocab, stream=s)
    torch.cuda.synchronize()
    for b in (got, other):
        for p, q in zip(b.outputs(), ref.outputs()):
            assert torch.equal(p, q)


def test_captured_replays():
    """Replays with new inputs and other counted tokens, two graphs on one workspace, eager work between them."""
    (x, w, y), vocab = make()
    sets = [Buffers(700, 256, 3000, "bf16") for _ in range(2)]
    sets[1].ws = sets[0].ws
    eager = Buffers(700, 256, 3000, "bf16")
    eager.step(x, w, y, vocab)
    graphs = []
    for b in sets:
        b.step(x, w, y, vocab)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.step(x, w, y, vocab)
        graphs.append(g)
    for i in range(4):
        (nx, nw, ny), _ = make(seed=20 + i)
        x.copy_(nx), w.copy_(nw), y.copy_(ny)
        if i == 2:
            y.fill_(-100)
        for b in sets:
            for t in b.outputs():
                t.fill_(3)
        eager.step(x, w, y, vocab)
        graphs[i % 2].replay()
        graphs[1 - i % 2].replay()
        torch.cuda.synchronize()
        for b in sets:
            for p, q in zip(b.outputs(), eager.outputs()):
                assert torch.equal(p, q), i


def test_more_than_2_to_31_logits():
    """65536 x 40000: offsets past 32 bits in the statistics; losses of a few tokens, counted by a rule."""
    T, H, V = 65536, 8, 40000
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = torch.randn(H, V, generator=g, device="cuda").bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    b = Buffers(T, H, V, "bf16")
    b.step(x, w, y, V)
    torch.cuda.synchronize()
    for t in (0, 255, 256, 40000, T - 1):
        l = x[t].double() @ w.double()
        lse = torch.logsumexp(l, 0)
        assert abs(float(b.lse[t]) - float(lse)) <= 1e-4 and abs(float(b.loss[t]) - float(lse - l[y[t]])) <= 2e-4
        p = torch.exp(l - lse)
        p[y[t]] -= 1
        want, size = w.double() @ p / T, w.double().abs() @ p.abs() / T
        assert ((b.dx[t].double() - want).abs() <= 2.0 ** -7 * size).all()
