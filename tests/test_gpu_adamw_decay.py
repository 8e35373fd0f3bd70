"""Weight decay and steps far below a weight's own precision: what the 64-bit formula
takes off arrives, to the state's own rounding where that is to nearest, and in the
mean where weights are rounded by hash."""
import numpy as np
import pytest
import torch

import step_ref as S
from block_ref import U, host
from expert_grouped_gemm_top_amd import moe

pytestmark = pytest.mark.gpu


def tensor(w, dtype, bits, master, decay, grad=None):
    n, z = w.numel(), lambda d, k: torch.zeros(k, dtype=d, device="cuda")  # noqa: E731
    extra = dict(m_scale=z(torch.float32, -(-n // 256)), v_scale=z(torch.float32, -(-n // 256))) if bits == 8 else {}
    if master:
        extra["master"] = w.clone()
    d = torch.uint8 if bits == 8 else torch.float32
    p = w.to(dtype, copy=True)
    return moe.AdamWTensor(p, torch.zeros_like(p) if grad is None else grad.to(dtype), z(d, n), z(d, n), weight_decay=decay, **extra)


def steps(t, lr, k, seed=3):
    counter, rate = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.full((1,), lr, device="cuda")
    plan = moe.AdamWPlan([t])
    for _ in range(k):
        moe.moe_adamw_step(plan, counter, rate, seed=seed)
    torch.cuda.synchronize()


# n bf16 weights in [1, 2), steps of 2^-7 (the 1 itself 2^-8 below it).  A step of the optimizer takes a weight down by a
# whole one with the probability (lr decay p) / 2^-7: the mean of n after k steps has a deviation of at most
# sqrt(k lr decay 2 2^-7 / n), six of which are allowed, beside a mean that is k lr decay of the weights'.
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lr,decay", [(1e-6, 0.1), (2e-5, 0.01), (1e-6, 0.01), (1e-3, 0.1)])
@pytest.mark.parametrize("ones", [False, True])
def test_bf16_weights_decay_in_the_mean(lr, decay, bits, ones):
    n, k = 1 << 24, 400
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.ones(n, device="cuda") if ones else (1 + torch.randint(0, 128, (n,), generator=g, device="cuda") / 128.0)
    w[::2] *= -1
    t = tensor(w, torch.bfloat16, bits, False, decay)
    before = float(t.param.double().abs().mean())
    steps(t, lr, k)
    rate = float(np.float32(lr)) * decay
    want = before * -np.expm1(k * np.log1p(-rate))
    assert abs(before - float(t.param.double().abs().mean()) - want) <= 6 * (k * rate * 2 * 2.0 ** -7 / n) ** 0.5 + 2.0 ** -23 * want


@pytest.mark.parametrize("bits", [32, 8])
def test_bf16_weights_that_nothing_moves_stay(bits):
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn(1 << 20, device="cuda", generator=g)
    w[:6] = torch.tensor([1.0, -2.0, 0.0, -0.0, 2.0 ** -126, 2.0 ** -133])
    t = tensor(w, torch.bfloat16, bits, False, 0.0)
    before = t.param.clone()
    steps(t, 1.0, 20)
    assert torch.equal(before.view(torch.int16), t.param.view(torch.int16))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,master", [(torch.float32, False), (torch.bfloat16, True)])
@pytest.mark.parametrize("lr,decay", [(1e-6, 0.1), (2e-5, 0.01), (1e-6, 0.01), (0.5, 0.5)])
@pytest.mark.parametrize("moved", [False, True])
def test_fp32_weights_are_off_by_their_own_rounding(dtype, master, lr, decay, bits, moved):
    """Half a step of the result, 2^-24 of it, and of the decrement its own roundings: four for the decay, sixteen for the
    update (as in step_ref.adamw), where m's terms do not cancel (m was 0)."""
    n = 1 << 16
    g = torch.Generator(device="cuda").manual_seed(3)
    w = 0.02 * torch.randn(n, device="cuda", generator=g)
    grad = torch.randn(n, device="cuda", generator=g) if moved else None
    t = tensor(w, dtype, bits, master, decay, grad)
    steps(t, lr, 1)
    a, r = host(w), float(np.float32(lr))
    p, _, _, _ = S.adamw(a, 0.0 * a if grad is None else host(t.grad), 0.0, 0.0, 1, r, 0.9, 0.999, 1e-8, decay, 1.0)
    got = host(t.master if master else t.param)
    took = r * decay * np.abs(a)
    err = U["f32"] * (np.abs(p) + 4 * took + 20 * np.abs(p - a * (1 - r * decay)))
    assert (np.abs(got - p) <= err).all(), np.max(np.abs(got - p) - err)


def test_shares_below_2_to_16_of_a_step():
    """A decrement of 2^-24 of a step of weights that are 1: the formula's share of them goes down, by the hash that the
    header states: those whose 32 bits are below it."""
    n = 1 << 24  # the first step of equal gradients is lr, beside steps of 2^-8 below 1
    for shift, k in ((24, 1), (18, 1), (12, 2)):
        lr = 2.0 ** (-8 - shift)
        w = torch.ones(n, device="cuda")
        t = tensor(w, torch.bfloat16, 32, False, 0.0, torch.ones(n, device="cuda"))
        steps(t, lr, 1, seed=k)
        r = S.dither(0, n, 1, k) * np.uint64(0x9e3779b1) & np.uint64(0xffffffff)
        down = t.param.float().cpu().numpy() != 1
        # the update is lr to within 2^-20 of it, and so is the border
        sure = np.abs(r.astype(np.float64) - 2.0 ** (32 - shift)) > 2.0 ** (32 - shift - 20) + 1
        assert np.array_equal(down[sure], (r < 2 ** (32 - shift))[sure]), shift
        assert shift > 18 or down.any()  # 64 are expected of 2^-18, one of 2^-24
        assert (t.param[torch.from_numpy(down).cuda()] == 1 - 2.0 ** -8).all()


@pytest.mark.parametrize("shift,fine", [(11, False), (12, False), (14, True), (16, True)])
def test_shares_of_16_and_of_32_bits(shift, fine):
    """Weights of 1 that go down by 2^-shift and 2^-25 more: 2^(8 - shift) of a step of 2^-8, and 2^-17.  Of those whose
    h >> 16 is at that border, half go down by 32 bits, and by 16 all or none."""
    n, k = 1 << 24, 4
    t = tensor(torch.ones(n, device="cuda"), torch.bfloat16, 32, False, 0.0, torch.ones(n, device="cuda"))
    steps(t, 2.0 ** -shift + 2.0 ** -25, 1, seed=k)
    h = (S.dither(0, n, 1, k) * np.uint64(0x9e3779b1) & np.uint64(0xffffffff)).astype(np.int64)
    down, border = t.param.float().cpu().numpy() != 1, 1 << (24 - shift)
    assert np.array_equal(down[h >> 16 != border], (h >> 16 < border)[h >> 16 != border])
    at = h >> 16 == border
    assert at.sum() > 100
    if fine:  # the update is lr to 2^-20 of it
        sure = at & (np.abs((h & 0xffff) - 2 ** 15) > 2.0 ** (32 + 8 - shift - 20) + 1)
        assert np.array_equal(down[sure], ((h & 0xffff) < 2 ** 15)[sure]) and sure.sum() > 50
    else:
        assert down[at].all() or not down[at].any()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,master", [(torch.float32, False), (torch.bfloat16, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_infinite_weights_stay(dtype, master, bits, decay):
    w = torch.full((300,), 0.5, device="cuda")
    w[3], w[299] = float("inf"), -float("inf")
    t = tensor(w, dtype, bits, master, decay, torch.ones(300, device="cuda"))
    steps(t, 1e-3, 2)
    p = t.param.float()
    assert p[3] == float("inf") and p[299] == -float("inf") and int(torch.isfinite(p).sum()) == 298
    if master:
        assert t.master[3] == float("inf") and t.master[299] == -float("inf")
