"""A training step with everything behind the block: block with balance loss, head
with the vocabulary loss, both backward, AdamW.  Values and gradients against
float64 autograd, the update against the 64-bit step, whole steps captured."""
import numpy as np
import pytest
import torch

import block_ref as R
import step_ref as S
from expert_grouped_gemm_top_amd import moe
from expert_grouped_gemm_top_amd.layer import AdamWBuffers, BalanceLoss, MoeBlockBuffers, MoeHeadBuffers, MoeLayerBuffers, ScoredRouting
from moe_cases import note

pytestmark = pytest.mark.gpu

ROUTINGS = [ScoredRouting(moe.MOE_SCORE_SIGMOID, 4, 2, 2, True, 2.5), ScoredRouting(moe.MOE_SCORE_SOFTMAX, renormalize=False)]
H, F, E, K, SH, V, VOCAB = 128, 64, 16, 4, 96, 520, 515
DECAY = dict.fromkeys(("w_r", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down", "head"), 0.1)


def parameters(dtype, seed):
    rng = np.random.default_rng(seed)
    r = lambda scale, *s: R.rounded(scale * rng.standard_normal(s), dtype)  # noqa: E731
    return dict(gamma=R.rounded(1 + 0.25 * rng.standard_normal(H), dtype), beta=r(0.25, H), w_r=r(H ** -0.5, H, E),
                w_gate=r(H ** -0.5, E, H, F), w_up=r(H ** -0.5, E, H, F), w_down=r(F ** -0.5, E, F, H),
                s_gate=r(H ** -0.5, H, SH), s_up=r(H ** -0.5, H, SH), s_down=r(SH ** -0.5, SH, H), head=r(2 * H ** -0.5, H, V))


class Step:
    """The buffers of a step over T tokens, and its calls."""

    def __init__(self, T, p, dtype, routing, offsets, bits=32, master=False, device_params=None):
        d = R.DT[dtype]
        self.p = device_params or {n: R.dev(a, dtype) for n, a in p.items()}
        self.offsets = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
        self.block = MoeBlockBuffers(T, H, F, E, K, SH, routing, d, balance=BalanceLoss(0.5, 1 if offsets is None else len(offsets) - 1))
        self.head = MoeHeadBuffers(T, H, V, VOCAB, d)
        self.grads = dict(self.block.grads, head=self.head.dw)
        self.opt = AdamWBuffers(self.p, self.grads, 1e-3, DECAY, bits=bits, master=master, seed=3)

    def forward_backward(self, x, y, stream=None):
        h = self.block.forward(x, self.p, stream, self.offsets)
        self.head.forward(h, self.p["head"], y, stream)
        dy = self.head.backward(h, self.p["head"], y, stream=stream)
        self.block.backward(dy, self.p, stream=stream)

    def __call__(self, x, y, stream=None):
        self.forward_backward(x, y, stream)
        self.opt.step(stream=stream)

    def outputs(self):
        L = self.block.layer
        states = {f"{n}.{k}": t for n, s in self.opt.state.items() for k, t in s.items()}
        return {**self.grads, **{"new " + n: t for n, t in self.p.items()}, **states, "loss": self.head.loss, "mean": self.head.mean,
                "balance": L.balance_loss, "counts": L.balance_counts, "dx": self.block.dx}


def autograd_step(x, y, p, idx, counts, routing, offsets, eps):
    """Losses and gradients in float64 for the selection and counts that were made."""
    t = {n: torch.from_numpy(a).requires_grad_() for n, a in p.items()}
    xt = torch.from_numpy(x).requires_grad_()
    xn = torch.nn.functional.layer_norm(xt, (H,), t["gamma"], t["beta"], eps)
    logits = xn @ t["w_r"]
    s = torch.softmax(logits, 1) if routing.score == 0 else torch.sigmoid(logits)
    sel = torch.from_numpy(idx.astype(np.int64))
    w = s.gather(1, sel)
    w = routing.scale * (w / w.sum(1, keepdim=True) if routing.renormalize else w)
    rows = []
    for i in range(x.shape[0]):
        e = sel[i]
        h = torch.nn.functional.silu(xn[i] @ t["w_gate"][e]) * (xn[i] @ t["w_up"][e])
        rows.append((w[i][:, None] * torch.einsum("kf,kfh->kh", h, t["w_down"][e])).sum(0))
    out = torch.nn.functional.silu(xn @ t["s_gate"]) * (xn @ t["s_up"]) @ t["s_down"] + torch.stack(rows)
    share, seq = s / s.sum(1, keepdim=True), S.sequences(len(x), offsets)
    n = (seq >= 0).sum()
    balance = sum(0.5 * E / K / n * (torch.from_numpy(counts[i].astype(np.float64)) * share[seq == i].mean(0)).sum()
                  for i in range(len(offsets) - 1) if (seq == i).any())
    target = torch.from_numpy(np.where((y >= 0) & (y < VOCAB), y, -100).astype(np.int64))
    ce = torch.nn.functional.cross_entropy(out @ t["head"][:, :VOCAB], target)
    names = list(t)
    g = torch.autograd.grad(ce + balance, [xt] + [t[n] for n in names])
    return ce.item(), balance.item(), g[0].numpy(), dict(zip(names, (a.numpy() for a in g[1:])))


# Relative to each tensor's largest value, as for the block alone: fp32 eight products in a row, each off by at most
# 256 2^-24 of its terms' sizes; bf16 at most fourteen stored values in a row, each off by at most 2^-8.
TOL = {"f32": 8 * 256 * 2.0 ** -24, "bf16": 14 * 2.0 ** -8}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("routing", [0, 1])
@pytest.mark.parametrize("bits", [32, 8])
def test_step_matches_autograd_and_the_update(dtype, routing, bits):
    T, offsets = 77, [0, 20, 20, 70]
    routing = ROUTINGS[routing]
    note(f"train step {dtype} {routing} {bits}")
    p = parameters(dtype, 31)
    rng = np.random.default_rng(32)
    x, y = R.rounded(rng.standard_normal((T, H)), dtype), rng.integers(0, VOCAB, T).astype(np.int32)
    y[rng.random(T) < 0.3] = -100
    master = dtype == "bf16" and bits == 32
    step = Step(T, p, dtype, routing, offsets, bits, master)
    step(R.dev(x, dtype), torch.from_numpy(y).cuda())
    torch.cuda.synchronize()
    L = step.block.layer
    idx, counts = L.topk_idx.cpu().numpy(), L.balance_counts.cpu().numpy()
    ce, balance, dx, grads = autograd_step(x, y, p, idx, counts, routing, offsets, step.block.eps)
    assert abs(float(step.head.mean[0]) - ce) <= TOL[dtype] * ce and abs(float(L.balance_loss) - balance) <= TOL[dtype] * balance
    for name, got, ref in [("dx", step.block.dx, dx)] + [(n, step.grads[n], g) for n, g in grads.items()]:
        err = np.abs(R.host(got) - ref).max() / np.abs(ref).max()
        assert err <= TOL[dtype], f"{name}: {err:.3e}"
    block = 0
    for name, a in p.items():  # the update from the gradients that are there
        g, w = R.host(step.grads[name]).reshape(-1), a.reshape(-1)
        ref, _, _, err = S.adamw(w, g, 0.0, 0.0, 1, float(np.float32(1e-3)), 0.9, 0.999, 1e-8, DECAY.get(name, 0.0), 1.0)
        new = R.host(step.p[name]).reshape(-1)
        if dtype == "f32":
            assert (np.abs(new - ref) <= err).all(), name
        else:  # rounded to nearest from a master, or to one of the two neighbours
            gap = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(ref), 2.0 ** -126))) - 7)
            assert (np.abs(new - ref) <= (0.5 * gap if master else gap) + 2 * err).all(), name
        block += -(-len(g) // 256)
    assert step.opt.counter.tolist() == [1, 0]


def test_plain_routing_with_a_balance_loss():
    """A layer without scored routing: its router's gradient with alpha 0 is moe_router_bwd's, with alpha it has the loss'."""
    T = 60
    rng = np.random.default_rng(5)
    w = {n: R.dev(a, "f32") for n, a in parameters("f32", 33).items()}
    x, dy = (R.dev(rng.standard_normal((T, H)), "f32") for _ in range(2))

    def run(balance):
        L = MoeLayerBuffers(T, H, F, E, K, torch.float32, router=True, balance=balance)
        L.forward(None, x, w["w_gate"], w["w_up"], w["w_down"], w_r=w["w_r"])
        L.backward(dy, w["w_gate"], w["w_up"], w["w_down"], w_r=w["w_r"])
        torch.cuda.synchronize()
        return L

    plain, zero, full = run(None), run(BalanceLoss(0.0)), run(BalanceLoss(3.0))
    # either form of the selected softmax' gradient: k differences of fp32 values, 16 2^-24 of the largest
    assert (plain.dlogits - zero.dlogits).abs().max() <= 16 * 2.0 ** -24 * plain.dlogits.abs().max()
    l = R.host(full.logits)
    ref, size = S.balance_bwd(l, full.balance_counts.cpu().numpy(), K, [0, T], 0, 3.0, 1.0)
    off = np.abs(R.host(full.dlogits) - R.host(zero.dlogits) - ref)
    assert (off <= (4 * np.abs(l).max() + 60) * 3 * 2.0 ** -23 * size + 2.0 ** -22 * np.abs(R.host(full.dlogits))).all()


def test_a_balance_loss_that_would_be_lost_is_refused():
    """One of other logits than the router's, sequences without a loss, a gradient that nothing takes."""
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    ws, x = (f(E, H, F), f(E, H, F), f(E, F, H)), f(8, H)
    offsets = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    with_loss, without = (MoeLayerBuffers(8, H, F, E, K, torch.float32, router=True, balance=b) for b in (BalanceLoss(1.0), None))
    for call in (lambda: with_loss.forward(f(8, E), x, *ws), lambda: without.forward(None, x, *ws, w_r=f(H, E), seq_offsets=offsets),
                 lambda: without.backward(x, *ws, w_r=f(H, E), dbalance=f(1)), lambda: with_loss.backward(x, *ws, dbalance=f(1)),
                 lambda: MoeLayerBuffers(8, H, F, E, K, torch.float32, balance=BalanceLoss(1.0))):
        with pytest.raises(AssertionError, match="balance"):
            call()


def batch(T, seed):
    rng = np.random.default_rng(seed)
    y = rng.integers(0, VOCAB, T).astype(np.int32)
    y[rng.random(T) < 0.3] = -100
    return R.dev(rng.standard_normal((T, H)), "bf16"), torch.from_numpy(y).cuda()


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_training_steps(bits):
    """Replays train on as eager steps do, bit for bit, with eager work between them."""
    T, offsets, p = 1100, [0, 500, 1090], parameters("bf16", 41)
    eager, captured = (Step(T, p, "bf16", ROUTINGS[0], offsets, bits, bits == 32) for _ in range(2))
    x, y = batch(T, 50)
    for s in (eager, captured):
        s.forward_backward(x, y)  # what a first call sets up
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured(x, y)
    for i in range(4):
        nx, ny = batch(T, 60 + i)
        x.copy_(nx), y.copy_(ny)
        for s in (eager, captured):
            s.opt.lr.fill_(1e-3 / (i + 1))
        g.replay()
        eager(x, y)
        torch.cuda.synchronize()
        ref = eager.outputs()
        for n, t in captured.outputs().items():
            assert torch.equal(t, ref[n]), (i, n)
    assert captured.opt.counter.tolist() == [4, 0]


def test_two_trainings_at_once_on_other_streams():
    T, steps, refs = 300, [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in (71, 72):
        p = parameters("bf16", seed)
        steps.append((Step(T, p, "bf16", ROUTINGS[1], None, 8), Step(T, p, "bf16", ROUTINGS[1], None, 8), batch(T, seed)))
    torch.cuda.synchronize()
    for _ in range(3):
        for (a, b, data), s in zip(steps, streams):
            b(*data, stream=s)
    torch.cuda.synchronize()
    for a, b, data in steps:
        for _ in range(3):
            a(*data)
        torch.cuda.synchronize()
        ref = a.outputs()
        for n, t in b.outputs().items():
            assert torch.equal(t, ref[n]), n


def test_a_batch_of_which_nothing_is_counted():
    """No token is counted: zeros, not NaN, and the head stays but for its decay."""
    p = parameters("f32", 81)
    step = Step(40, p, "f32", ROUTINGS[1], [0, 0], 32)
    x, y = R.dev(np.random.default_rng(1).standard_normal((40, H)), "f32"), torch.full((40,), -100, dtype=torch.int32, device="cuda")
    step(x, y)
    torch.cuda.synchronize()
    assert step.head.mean.tolist() == [0.0, 0.0] and float(step.block.layer.balance_loss) == 0.0
    for n, g in step.grads.items():
        assert (g == 0).all(), n
    assert (np.abs(R.host(step.p["head"]) - p["head"] * (1 - np.float32(1e-3) * 0.1)) <= 2.0 ** -23 * np.abs(p["head"])).all()
