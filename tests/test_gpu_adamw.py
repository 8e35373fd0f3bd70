"""AdamW over many tensors against the 64-bit step: values, codes and scales, sizes
around the kernel's blocks, steps in a row, what is not finite, the rounding by
hash, captured steps, and what a plan refuses."""
import numpy as np
import pytest
import torch

import step_ref as S
from block_ref import DT, U, host, rounded
from expert_grouped_gemm_top_amd import moe
from moe_cases import note

pytestmark = pytest.mark.gpu

SIZES = [0, 1, 7, 8, 9, 255, 256, 257, 0, 2047, 2048, 2049, 5000, 100003]
B1, B2, EPS = 0.9, 0.999, 1e-8


def gpu(a, dt=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda()


def fp32(a):
    return np.asarray(a, np.float32).astype(np.float64)


class Model:
    """Tensors of a plan on both sides."""

    def __init__(self, sizes, dtype, bits, master, seed=0, fresh=False):
        rng = np.random.default_rng(seed)
        self.dtype, self.bits, self.master, self.sizes = dtype, bits, master, sizes
        self.p, self.m, self.v, self.t = [], [], [], []
        for i, n in enumerate(sizes):
            w = fp32(0.02 * rng.standard_normal(n))
            p = rounded(w, dtype)
            size = np.exp(2 * rng.standard_normal(n))
            m = 0 * w if fresh else fp32(3e-4 * size * rng.standard_normal(n))
            v = 0 * w if fresh else fp32(1e-6 * size * size)
            extra = {}
            if bits == 8:
                (mc, ms), (vc, vs) = S.codes(m, "m", 0.5), S.codes(v, "v", 0.5)
                if fresh:
                    mc, ms, vc, vs = (np.zeros_like(a) for a in (mc, ms, vc, vs))
                m, v = S.values(mc, ms, "m"), S.values(vc, vs, "v")
                extra = dict(m_scale=gpu(ms), v_scale=gpu(vs))
                state = gpu(mc, torch.uint8), gpu(vc, torch.uint8)
            else:
                state = gpu(m), gpu(v)
            if master:
                extra["master"] = gpu(w)
                p = w
            self.p.append(p)
            self.m.append(m)
            self.v.append(v)
            self.t.append(moe.AdamWTensor(gpu(rounded(w, dtype), DT[dtype]), torch.empty(n, dtype=DT[dtype], device="cuda"), *state,
                                          weight_decay=0.1 * (i % 3), **extra))
        self.plan = moe.AdamWPlan(self.t)
        self.counter = torch.zeros(2, dtype=torch.int32, device="cuda")
        self.lr = torch.full((1,), 1e-3, device="cuda")
        self.rng, self.steps = rng, 0

    def gradients(self):
        out = []
        for t, n in zip(self.t, self.sizes):
            g = rounded(1e-3 * np.exp(1.5 * self.rng.standard_normal(n)) * self.rng.standard_normal(n), self.dtype)
            t.grad.copy_(gpu(g, DT[self.dtype]))
            out.append(g)
        return out

    def step(self, seed, gs=None, check=True):
        grads = self.gradients()
        scale = None if gs is None else torch.tensor([gs], device="cuda")
        before = moe.moe_launch_count()
        moe.moe_adamw_step(self.plan, self.counter, self.lr, B1, B2, EPS, scale, seed)
        assert moe.moe_launch_count() - before == 1
        torch.cuda.synchronize()
        self.steps += 1
        assert self.counter.tolist() == [self.steps, 0]
        block = 0
        for i, (t, g) in enumerate(zip(self.t, grads)):
            lr = float(np.float32(1e-3))
            p, m, v, err = S.adamw(self.p[i], g, self.m[i], self.v[i], self.steps, lr, B1, B2, EPS, t.weight_decay,
                                   1.0 if gs is None else float(np.float32(gs)))
            r = S.dither(block, len(g), self.steps, seed)
            block += -(-len(g) // 256)
            self.compare(i, t, g, p, m, v, err, r, 1.0 if gs is None else gs)

    def compare(self, i, t, g, p, m, v, err, r, gs):
        name = f"tensor {i} of {len(g)}"
        if self.bits == 32:
            # four roundings of the terms' sizes each
            assert (np.abs(host(t.m) - m) <= 4 * U["f32"] * (np.abs(B1 * self.m[i]) + np.abs(0.1 * g * gs)) + 1e-44).all(), name
            assert (np.abs(host(t.v) - v) <= 6 * U["f32"] * v + 1e-44).all(), name
            self.m[i], self.v[i] = host(t.m), host(t.v)
        else:
            (mc, ms), (vc, vs) = S.codes(m, "m", ((r & np.uint64(0xffff)).astype(float) + 1 / 3) / 65536), \
                S.codes(v, "v", ((r >> np.uint64(16)).astype(float) + 1 / 3) / 65536)
            got = [x.cpu().numpy() for x in (t.m, t.m_scale, t.v, t.v_scale)]
            for a, b, what in zip(got, (mc, ms, vc, vs), ("m", "m_scale", "v", "v_scale")):
                assert np.array_equal(a & 127 if what == "m" else a, b & 127 if what == "m" else b), (name, what)
            assert (((got[0] ^ mc) & 128 == 0) | (mc & 127 == 0)).all(), name
            self.m[i], self.v[i] = S.values(got[0], ms, "m"), S.values(vc, vs, "v")
            if len(g):
                mo, vo = torch.empty(len(g), device="cuda"), torch.empty(len(g), device="cuda")
                moe.moe_adamw_moments(t.m, t.v, t.m_scale, t.v_scale, mo, vo)
                with np.errstate(under="ignore"):
                    assert np.array_equal(host(mo), self.m[i].astype(np.float32)) and np.array_equal(host(vo), self.v[i].astype(np.float32)), name
        if self.master:
            got = host(t.master)
            assert (np.abs(got - p) <= err).all(), name
            assert np.array_equal(host(t.param), rounded(got, self.dtype)), name
        elif self.dtype == "f32":
            got = host(t.param)
            assert (np.abs(got - p) <= err).all(), name
        else:
            got = host(t.param)
            gap = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(p), 2.0 ** -126))) - 7)
            left = np.abs(p) / gap - np.floor(np.abs(p) / gap)
            share = (((r * np.uint64(0x9e3779b1)) & np.uint64(0xffffffff)) >> np.uint64(16)).astype(float) / 65536
            # the kernel truncates an fp32 value: borders as far off as its error, and half an fp32 step
            near = err / gap + 2.0 ** -17
            sure = (np.abs(left + share - 1) > near) & (left > near) & (left < 1 - near)
            want = (np.floor(np.abs(p) / gap) + (left + share >= 1)) * gap * np.sign(p)
            assert np.array_equal(got[sure], want[sure]), name
            assert (np.abs(got - p) <= gap + err).all(), name
            assert len(g) < 100 or sure.mean() > 0.9
        self.p[i] = got


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,master", [("f32", False), ("bf16", False), ("bf16", True)])
def test_steps_in_a_row(dtype, master, bits):
    note(f"adamw {dtype} master={master} bits={bits}")
    m = Model(SIZES, dtype, bits, master)
    for seed, gs in ((5, None), (5, 0.7), (0xfffffff0, None)):
        m.step(seed, gs)


@pytest.mark.parametrize("bits", [32, 8])
def test_from_fresh_states(bits):
    """States of zeros (codes and scales) and the first steps' large bias corrections."""
    m = Model([300, 1, 4097], "f32", bits, False, seed=1, fresh=True)
    for i in range(3):
        m.step(i)


def test_many_tensors_and_one_large():
    m = Model([int(1 + (i * 7919) % 900) for i in range(700)] + [1 << 20], "bf16", 8, False, seed=2)
    m.step(9, 0.5)


def test_scales_at_their_borders():
    """Largest values at, just below and just above 448 and 1.75 times a power of two, and tiny and huge blocks."""
    n = 256 * 24
    a = np.zeros(n)
    tops = [448.0, np.nextafter(np.float32(448), np.float32(0)), np.nextafter(np.float32(448), np.float32(1e9)), 1.75, 1e-30, 1e-38,
            1e-42, 3e38, 2.0 ** -126, 0.0, 7.0, 224.0]
    for b, t in enumerate(tops * 2):
        a[256 * b:256 * (b + 1)] = np.float64(np.float32(t)) * np.linspace(0, 1, 256)
    g = gpu(a)
    p = torch.zeros(n, device="cuda")
    z8 = lambda: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    zs = lambda: torch.zeros(n // 256, device="cuda")  # noqa: E731
    t = moe.AdamWTensor(p, g, z8(), z8(), zs(), zs())
    plan, counter = moe.AdamWPlan([t]), torch.zeros(2, dtype=torch.int32, device="cuda")
    moe.moe_adamw_step(plan, counter, torch.zeros(1, device="cuda"), beta1=0.0, beta2=0.0, seed=3)
    torch.cuda.synchronize()
    r = S.dither(0, n, 1, 3)
    x = host(g)
    for got, scale, want in ((t.m, t.m_scale, S.codes(x, "m", ((r & np.uint64(0xffff)).astype(float) + 1 / 3) / 65536)),
                             (t.v, t.v_scale, S.codes(x * x, "v", ((r >> np.uint64(16)).astype(float) + 1 / 3) / 65536))):
        assert np.array_equal(scale.cpu().numpy(), want[1])
        keep = np.repeat(want[1] < 2.0 ** 127, 256)  # past it codes saturate
        assert np.array_equal(got.cpu().numpy()[keep], want[0][keep])
        assert (got.cpu().numpy()[~keep] <= 254).all()
    assert (p == 0).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_what_is_not_finite_stays_where_it_is(bits):
    m = Model([600], "f32", bits, False, seed=4)
    g = m.gradients()[0]
    bad = [0, 300, 301, 599]
    t = m.t[0]
    t.grad[bad] = torch.tensor([float("nan"), float("inf"), -float("inf"), float("nan")], device="cuda")
    moe.moe_adamw_step(m.plan, m.counter, m.lr)
    t.grad.copy_(gpu(g))
    moe.moe_adamw_step(m.plan, m.counter, m.lr)
    torch.cuda.synchronize()
    ok = np.delete(np.arange(600), bad)
    assert np.isfinite(host(t.param)[ok]).all() and not np.isfinite(host(t.param)[[0, 599]]).any()
    if bits == 8:
        assert (t.m.cpu().numpy()[bad] & 127 == 127).all() and (t.v.cpu().numpy()[bad] == 255).all()
        assert (t.m.cpu().numpy()[ok] & 127 != 127).all() and (t.v.cpu().numpy()[ok] != 255).all()
        assert np.isfinite(host(t.m_scale)).all() and np.isfinite(host(t.v_scale)).all()


def test_moments_in_8_bits_follow_the_mean():
    """v rounded by hash follows its average where rounding to nearest would stand still.  With g^2 = 1 from v = 4 on, the
    average after k steps is 1 + 3 b2^k.  A rounding is off by at most a step, 2^-3 of v below; independent, the average
    over n elements of their sum is off by sqrt(k / n) 2^-3 4 in the root mean square: six of those are allowed."""
    n, k = 1 << 16, 400
    t = moe.AdamWTensor(torch.zeros(n, device="cuda"), torch.ones(n, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda"),
                        gpu(S.codes(np.full(n, 4.0), "v", 0.5)[0], torch.uint8), torch.zeros(n // 256, device="cuda"),
                        gpu(S.codes(np.full(n, 4.0), "v", 0.5)[1]))
    plan, counter, lr = moe.AdamWPlan([t]), torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda")
    for _ in range(k):
        moe.moe_adamw_step(plan, counter, lr, seed=11)
    m, v = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    moe.moe_adamw_moments(t.m, t.v, t.m_scale, t.v_scale, m, v)
    assert abs(float(v.double().mean()) - (1 + 3 * B2 ** k)) <= 6 * (k / n) ** 0.5 * 0.5
    assert abs(float(m.double().mean()) - (1 - B1 ** k)) <= 6 * (k / n) ** 0.5 * 0.125


def test_bf16_weights_without_a_master_move():
    """Updates far below half a bf16 step arrive in the mean: 64 of 2^-16 on a weight of 1, whose steps are 2^-7 above
    and 2^-8 below.  Each rounding moves by at most a step; six deviations of the mean of n."""
    n, k = 1 << 16, 64
    t = moe.AdamWTensor(torch.ones(n, dtype=torch.bfloat16, device="cuda"), torch.ones(n, dtype=torch.bfloat16, device="cuda"),
                        torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"))
    plan, counter, lr = moe.AdamWPlan([t]), torch.zeros(2, dtype=torch.int32, device="cuda"), torch.full((1,), 2.0 ** -16, device="cuda")
    for _ in range(k):
        moe.moe_adamw_step(plan, counter, lr, seed=1)
    moved = 1.0 - float(t.param.double().mean())
    assert abs(moved - k * 2.0 ** -16) <= 6 * (k / n) ** 0.5 * 2.0 ** -7


def test_captured_steps_count_on():
    """Replays go on with the step count, the rate and the gradients that are there then."""
    a, b = Model([5000, 300], "bf16", 8, False, seed=6), Model([5000, 300], "bf16", 8, False, seed=6)
    scale = torch.ones(1, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_adamw_step(a.plan, a.counter, a.lr, grad_scale=scale, seed=2)
    for i in range(4):
        for t, u in zip(a.t, b.t):
            t.grad.normal_()
            u.grad.copy_(t.grad)
        a.lr.fill_(1e-3 / (i + 1))
        b.lr.copy_(a.lr)
        scale.fill_(1.0 / (i + 1))
        g.replay()
        moe.moe_adamw_step(b.plan, b.counter, b.lr, grad_scale=scale, seed=2)
        torch.cuda.synchronize()
        assert a.counter.tolist() == b.counter.tolist() == [i + 1, 0]
        for t, u in zip(a.t, b.t):
            for x, y in zip(t, u):
                if isinstance(x, torch.Tensor):
                    assert torch.equal(x, y)


def test_on_another_stream_and_two_at_once():
    models = [Model([70000, 5], "bf16", bits, False, seed=7) for bits in (8, 32)]
    refs = [Model([70000, 5], "bf16", bits, False, seed=7) for bits in (8, 32)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for m, r in zip(models, refs):
        m.gradients(), r.gradients()
        for _ in range(3):
            moe.moe_adamw_step(r.plan, r.counter, r.lr, seed=4)
    torch.cuda.synchronize()
    for _ in range(3):
        for m, s in zip(models, streams):
            moe.moe_adamw_step(m.plan, m.counter, m.lr, seed=4, stream=s)
    torch.cuda.synchronize()
    for m, r in zip(models, refs):
        for t, u in zip(m.t, r.t):
            assert torch.equal(t.param, u.param) and torch.equal(t.m, u.m) and torch.equal(t.v, u.v)


@pytest.mark.parametrize("bits", [32, 8])
def test_no_eps_and_gradients_whose_squares_are_subnormal(bits):
    """m / sqrt(v) is a sign where both decays are 0: of squares down to 2^-140, as fp32 keeps them (half a step of
    2^-149 of v, half of that of its root, and 16 roundings)."""
    g = np.array([2.0 ** -e * s * f for e in (30, 60, 62, 63, 64, 66, 68, 70) for s in (1, -1) for f in (1.0, 1.4)])
    n = len(g)
    for i in range(n) if bits == 8 else [slice(None)]:  # 8 bits: a block of its own for each
        a = np.atleast_1d(g[i])
        e = lambda dt=torch.float32: torch.zeros(len(a), dtype=dt, device="cuda")  # noqa: E731
        extra = dict(m_scale=e()[:1], v_scale=e()[:1]) if bits == 8 else {}
        d = torch.uint8 if bits == 8 else torch.float32
        t = moe.AdamWTensor(e(), gpu(a), e(d), e(d), **extra)
        c = torch.zeros(2, dtype=torch.int32, device="cuda")
        moe.moe_adamw_step(moe.AdamWPlan([t]), c, torch.ones(1, device="cuda"), 0.0, 0.0, 0.0)
        a = fp32(a)
        err = 16 * U["f32"] + 2.0 ** -150 / a ** 2
        assert (np.abs(host(t.param) + np.sign(a)) <= err).all(), (a, host(t.param))


@pytest.mark.parametrize("bits", [32, 8])
def test_tensors_past_32_bit_offsets(bits):
    """4.3e9 weights in one tensor and a small one behind it: their ends move as the formula says, the zeros between stay."""
    n = (1 << 32) + 4096 + 77 if bits == 8 else (1 << 31) + 4096 + 77
    h = torch.bfloat16
    z = lambda n, dt: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    d = torch.uint8 if bits == 8 else torch.float32
    make = lambda n: moe.AdamWTensor(z(n, h), z(n, h), z(n, d), z(n, d), **(  # noqa: E731
        dict(m_scale=z(-(-n // 256), torch.float32), v_scale=z(-(-n // 256), torch.float32)) if bits == 8 else {}))
    t, u = make(n), make(300)
    for a in (t, u):
        a.grad[-300:] = 0.5
        a.param[-300:] = 1.0
    t.grad[:300], t.param[:300] = 0.5, 1.0
    c = z(2, torch.int32)
    moe.moe_adamw_step(moe.AdamWPlan([t, u]), c, torch.full((1,), 0.125, device="cuda"), 0.5, 0.5, 0.0)
    torch.cuda.synchronize()
    # the first step of equal gradients is lr: 1 - 0.125, a bf16 value (or, from an fp32 one a rounding off, its neighbour)
    for a in (t.param[:300], t.param[-300:], u.param):
        assert (a.float() - 0.875).abs().max() <= 2.0 ** -8
        assert (a.float() == 0.875).float().mean() > 0.9
    for a in ([t.m[:300], t.m[-300:], u.m] if bits == 32 else []):
        assert (a == 0.25).all()
    if bits == 8:
        mo, vo = z(n, torch.float32), z(n, torch.float32)
        moe.moe_adamw_moments(t.m, t.v, t.m_scale, t.v_scale, mo, vo)
        for a in (slice(0, 300), slice(n - 300, n)):  # 0.25 and 0.125 are codes at their blocks' scales
            assert (mo[a] == 0.25).all() and (vo[a] == 0.125).all()
        assert int((t.m[300:-300] != 0).sum()) == 0
        del mo, vo
    # 0 / (0 + 0) is NaN with eps 0: the formula's
    assert torch.isnan(t.param[300:400]).all() and torch.isnan(t.param[-400:-300]).all()
    del t, u
    torch.cuda.empty_cache()


def test_nothing_to_do_is_a_step():
    t = Model([0, 0], "f32", 32, False)
    t.step(0)


def test_refusals():
    f = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    h = torch.bfloat16
    T = moe.AdamWTensor
    p = f(64)
    for bad, text in (([T(f(64), f(32), f(64), f(64))], "grad"), ([T(f(64), f(64, h), f(64), f(64))], "grad"),
                      ([T(f(64), f(64), f(64, h), f(64))], "m must"), ([T(f(64), f(64), f(64, torch.uint8), f(64, torch.uint8))], "m_scale"),
                      ([T(f(64), f(64), f(64), f(64), f(1), f(1))], "m_scale"), ([T(f(64), f(64), f(64), f(64), master=f(64))], "master"),
                      ([T(f(64), f(64), f(64), f(64)), T(f(64, h), f(64, h), f(64), f(64))], "param must"),
                      ([T(f(64, h), f(64, h), f(64), f(64), master=f(64)), T(f(64, h), f(64, h), f(64), f(64))], "master"),
                      ([T(p, p, f(64), f(64))], "overlaps"), ([T(f(65)[1:], f(64), f(64), f(64))], "aligned"),
                      ([T(f(64), f(64), f(64), f(64), weight_decay=float("nan"))], "weight_decay"), ([], "tensor"),
                      ([T(f(64).cpu(), f(64), f(64), f(64))], "param"), ([T(f(64, torch.float16), f(64), f(64), f(64))], "dtype")):
        with pytest.raises(moe.MoeError, match=text):
            moe.AdamWPlan(bad)
    plan = moe.AdamWPlan([T(f(64), f(64), f(64), f(64))])
    c = torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw, text in ((dict(beta1=1.0), "beta"), (dict(beta2=-0.1), "beta"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=1e-40), "eps"), (dict(eps=1e-300), "eps"), (dict(eps=1e38), "eps"),
                     (dict(grad_scale=f(2)), "grad_scale"), (dict(lr=f(2)), "lr"), (dict(lr=None), "lr"), (dict(counter=c[:1]), "counter")):
        with pytest.raises(moe.MoeError, match=text):
            moe.moe_adamw_step(plan, **{**dict(counter=c, lr=f(1)), **kw})
    assert c.tolist() == [0, 0]
