"""The operators of a MoE block together, as a training step runs them
(MoeBlockBuffers: layer norm, router, scored routing, routed experts, gated
shared expert): values and gradients against float64 autograd, on a stream of
its own, in captured graphs, and with the documented launch counts."""
import numpy as np
import pytest
import torch

import block_ref as R
from expert_grouped_gemm_top_amd import moe
from expert_grouped_gemm_top_amd.layer import MoeBlockBuffers, MoeLayerBuffers, ScoredRouting
from moe_cases import note

pytestmark = pytest.mark.gpu

ROUTINGS = [ScoredRouting(moe.MOE_SCORE_SIGMOID, 4, 2, 2, True, 2.5), ScoredRouting(moe.MOE_SCORE_SOFTMAX, renormalize=False),
            ScoredRouting(moe.MOE_SCORE_SOFTMAX, 4, 3, 1, True, 1.0)]


def params(H, F, E, S, dtype, seed, beta=True, bias=True):
    rng = np.random.default_rng(seed)
    r = lambda scale, *s: R.rounded(scale * rng.standard_normal(s), dtype)  # noqa: E731
    p = dict(gamma=1 + r(0.25, H), beta=r(0.25, H), w_r=r(H ** -0.5, H, E), w_gate=r(H ** -0.5, E, H, F),
             w_up=r(H ** -0.5, E, H, F), w_down=r(F ** -0.5, E, F, H), s_gate=r(H ** -0.5, H, S), s_up=r(H ** -0.5, H, S),
             s_down=r(S ** -0.5, S, H), route_bias=np.float64(np.float32(0.2 * rng.standard_normal(E))))
    p["gamma"] = R.rounded(p["gamma"], dtype)
    if not beta:
        p["beta"] = None
    if not bias:
        p["route_bias"] = None
    return p


def on_device(p, dtype):
    return {n: None if a is None else (torch.from_numpy(np.float32(a)).cuda() if n == "route_bias" else R.dev(a, dtype))
            for n, a in p.items()}


def autograd_block(x, p, idx, routing, dy, eps):
    """The block in float64 for the selection `idx`, and its gradients."""
    t = {n: torch.from_numpy(a).requires_grad_() for n, a in p.items() if a is not None and n != "route_bias"}
    xt = torch.from_numpy(x).requires_grad_()
    xn = torch.nn.functional.layer_norm(xt, (x.shape[1],), t["gamma"], t.get("beta"), eps)
    logits = xn @ t["w_r"]
    s = torch.softmax(logits, 1) if routing.score == moe.MOE_SCORE_SOFTMAX else torch.sigmoid(logits)
    w = s.gather(1, torch.from_numpy(idx.astype(np.int64)))
    if routing.renormalize:
        w = w / w.sum(1, keepdim=True)
    w = routing.scale * w
    y = torch.nn.functional.silu(xn @ t["s_gate"]) * (xn @ t["s_up"]) @ t["s_down"]
    rows = []
    for i in range(x.shape[0]):
        e = torch.from_numpy(idx[i].astype(np.int64))
        h = torch.nn.functional.silu((xn[i] @ t["w_gate"][e])) * (xn[i] @ t["w_up"][e])
        rows.append((w[i][:, None] * torch.einsum("kf,kfh->kh", h, t["w_down"][e])).sum(0))
    y = y + torch.stack(rows)
    names = list(t)
    grads = torch.autograd.grad(y, [xt] + [t[n] for n in names], torch.from_numpy(dy))
    return y.detach().numpy(), grads[0].numpy(), dict(zip(names, (g.numpy() for g in grads[1:]))), logits.detach().numpy()


# Relative to each tensor's largest value.  fp32: six products in a row, each off by at most 256 2^-24 of its
# terms' sizes.  bf16: at most ten stored values in a row (norm, pre-activation, hidden, output row, sum; the same on
# the way back), each off by at most 2^-8.
TOL = {"f32": 6 * 256 * 2.0 ** -24, "bf16": 10 * 2.0 ** -8}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("routing", range(3))
def test_block_matches_autograd(dtype, routing):
    T, H, F, E, k, S = 77, 128, 64, 16, 4, 96
    routing = ROUTINGS[routing]
    note(f"block {dtype} {routing}")
    p = params(H, F, E, S, dtype, 21, beta=routing.score == 1, bias=routing.score == 1)
    rng = np.random.default_rng(22)
    x, dy, skip = (R.rounded(rng.standard_normal((T, H)), dtype) for _ in range(3))
    d = on_device(p, dtype)
    B = MoeBlockBuffers(T, H, F, E, k, S, routing, R.DT[dtype])
    B.forward(R.dev(x, dtype), d)
    B.backward(R.dev(dy, dtype), d, dx_add=R.dev(skip, dtype))
    torch.cuda.synchronize()
    idx = B.layer.topk_idx.cpu().numpy()
    want = R.route(R.host(B.layer.logits), p["route_bias"], k, routing.score, routing.n_groups, routing.top_groups,
                   routing.group_top)[0]
    assert np.array_equal(idx, want)
    y, dx, grads, _ = autograd_block(x, p, idx, routing, dy, B.eps)
    for name, got, ref in [("y", B.y, y), ("dx", B.dx, dx + skip)] + [(n, B.grads[n], g) for n, g in grads.items()]:
        err = np.abs(R.host(got) - ref).max() / np.abs(ref).max()
        assert err <= TOL[dtype], f"{name}: {err:.3e}"


def make(T=300, H=256, F=128, E=32, k=4, S=192, seed=23):
    p = on_device(params(H, F, E, S, "bf16", seed), "bf16")
    B = MoeBlockBuffers(T, H, F, E, k, S, ROUTINGS[0])
    rng = np.random.default_rng(seed + 1)
    new = lambda: R.dev(rng.standard_normal((T, H)), "bf16")  # noqa: E731
    return B, p, new


def outputs(B):
    L = B.layer
    return {**B.grads, "y": B.y, "dx": B.dx, "topk_w": L.topk_w, "topk_idx": L.topk_idx, "dlogits": L.dlogits, "mean": B.mean}


def step(B, p, x, dy, stream=None):
    B.forward(x, p, stream)
    B.backward(dy, p, dx_add=dy, stream=stream)


def test_block_on_another_stream():
    """The same step on a stream that is not the current one, ordered behind the inputs by an event."""
    B, p, new = make()
    x, dy = new(), new()
    step(B, p, x, dy)
    torch.cuda.synchronize()
    ref = {n: t.clone() for n, t in outputs(B).items()}
    for t in outputs(B).values():
        t.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(B, p, x, dy, s)
    s.synchronize()
    for n, t in outputs(B).items():
        assert torch.equal(t, ref[n]), n


def test_two_blocks_at_once():
    """Two steps on two streams, each with its own buffers, interleaved call by call."""
    steps = []
    for seed in (23, 40):
        B, p, new = make(seed=seed)
        steps.append((B, p, new(), new()))
    ref = []
    for B, p, x, dy in steps:
        step(B, p, x, dy)
        torch.cuda.synchronize()
        ref.append({n: t.clone() for n, t in outputs(B).items()})
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for s, (B, p, x, dy) in zip(streams, steps):
            s.wait_stream(torch.cuda.current_stream())
            step(B, p, x, dy, s)
    torch.cuda.synchronize()
    for r, (B, *_) in zip(ref, steps):
        for n, t in outputs(B).items():
            assert torch.equal(t, r[n]), n


def test_block_in_a_captured_graph():
    """Replays with new inputs are the eager step bit for bit, with eager steps between them, and two graphs
    that share a workspace, replayed in turn."""
    B, p, new = make()
    B2 = MoeBlockBuffers(300, 256, 128, 32, 4, 192, ROUTINGS[0])
    B2.ws = B.ws
    x, dy = new(), new()
    step(B, p, x, dy)
    step(B2, p, x, dy)
    torch.cuda.synchronize()
    graphs = []
    for b in (B, B2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(b, p, x, dy)
        graphs.append(g)
    E = MoeBlockBuffers(300, 256, 128, 32, 4, 192, ROUTINGS[0])
    for i in range(4):
        note(f"replay {i}")
        x.copy_(new())
        dy.copy_(new())
        for b in (B, B2):
            for t in outputs(b).values():
                t.fill_(7)
        step(E, p, x, dy)
        graphs[i % 2].replay()
        graphs[1 - i % 2].replay()
        torch.cuda.synchronize()
        ref = {n: t.clone() for n, t in outputs(E).items()}
        for b in (B, B2):
            for n, t in outputs(b).items():
                assert torch.equal(t, ref[n]), (i, n)


def test_repeated_steps_are_bitwise_the_same():
    B, p, new = make(T=1030, seed=30)
    x, dy = new(), new()
    first = None
    for _ in range(3):
        step(B, p, x, dy)
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in outputs(B).items()}
        first = first or got
        for n in got:
            assert torch.equal(got[n], first[n]), n


def test_layer_without_scored_routing_takes_no_bias():
    L = MoeLayerBuffers(8, 64, 64, 8, 2)
    with pytest.raises(AssertionError):
        L.forward(torch.zeros(8, 8, device="cuda"), torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda"), None, None,
                  None, route_bias=torch.zeros(8, device="cuda"))


def counted(f, *a, **kw):
    before = moe.moe_launch_count()
    f(*a, **kw)
    return moe.moe_launch_count() - before


def test_launch_counts():
    T, E, k, H, O = 100, 32, 4, 256, 136  # noqa: E741
    f = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    b = lambda *s: f(*s, dt=torch.bfloat16)  # noqa: E731
    idx = f(T, k, dt=torch.int32)
    assert counted(moe.moe_route_scored, f(T, E), None, idx, f(T, k), k) == 1
    assert counted(moe.moe_route_scored_bwd, f(T, E), idx, f(T, k), f(T, E)) == 1
    assert counted(moe.moe_layernorm_fwd, b(T, H), b(H), None, b(T, H)) == 1
    ws = f(1 << 24, dt=torch.uint8)
    w, y = b(H, O), b(T, O)
    assert counted(moe.moe_linear_fwd, b(T, H), w, None, y, workspace=ws) == 1
    assert counted(moe.moe_linear_bwd, b(T, H), w, y, None, b(T, H), b(H, O), workspace=ws) == 1
    assert counted(moe.moe_linear_bwd, b(T, H), w, y, None, b(T, H), b(H, O), b(O), workspace=ws) == 2
    assert counted(moe.moe_linear_bwd, b(T, H), w, y, b(T, O), b(T, H), b(H, O), b(O), 4, y, workspace=ws) == 2
    # one row tile and a long reduction: split, so its slices are added
    assert counted(moe.moe_linear_fwd, b(8, 8192), b(8192, 64), None, b(8, 64), workspace=ws) == 2
    assert counted(moe.moe_layernorm_bwd, b(T, H), b(H), f(T), f(T), b(T, H), b(T, H), b(H), b(H), ws) == 2
    torch.cuda.synchronize()


def test_profiling_hook_times_the_new_phases():
    import ctypes
    L = moe.lib()
    L.moe_profile_kernel.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    B, p, new = make()
    x, dy = new(), new()
    step(B, p, x, dy)
    torch.cuda.synchronize()
    ref = {n: t.clone() for n, t in outputs(B).items()}
    events = {}
    for kind in (12, 13, 14, 15):  # MOE_K_ROUTE_SCORED, LAYERNORM, LINEAR_FWD, LINEAR_BWD
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record(), b.record()
        events[kind] = (a, b)
        assert L.moe_profile_kernel(kind, ctypes.c_void_p(a.cuda_event), ctypes.c_void_p(b.cuda_event)) == 0
    assert L.moe_profile_kernel(16, None, None) == 1
    step(B, p, x, dy)
    torch.cuda.synchronize()
    for kind, (a, b) in events.items():
        assert 0.0 < a.elapsed_time(b) < 50.0, kind
    for n, t in outputs(B).items():
        assert torch.equal(t, ref[n]), n


def test_calls_on_another_device_are_refused():
    """A tensor of a device that is not the current one (made up here: one GPU is enough)."""
    class Elsewhere(torch.Tensor):
        @property
        def device(self):
            return torch.device("cuda", torch.cuda.current_device() + 1)

        def get_device(self):
            return torch.cuda.current_device() + 1

    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(moe.MoeError, match="current device"):
        moe.moe_layernorm_fwd(x.as_subclass(Elsewhere), x[0].clone(), None, torch.empty_like(x))


def test_binding_refuses_wrong_shapes_and_types():
    x = torch.zeros(4, 64, device="cuda")
    h = x.bfloat16()
    g = x[0].clone()
    idx, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    for call in (lambda: moe.moe_layernorm_fwd(x, g[:32], None, x), lambda: moe.moe_layernorm_fwd(h, g, None, h),
                 lambda: moe.moe_layernorm_fwd(x.t(), g, None, x.t()), lambda: moe.moe_layernorm_fwd(x.double(), g, None, x),
                 lambda: moe.moe_layernorm_fwd(x[:, :56], g[:56], None, x[:, :56]),
                 lambda: moe.moe_route_scored(x, None, idx.long(), w, 2), lambda: moe.moe_route_scored(x, None, idx, w, 3),
                 lambda: moe.moe_route_scored(x, g[:8], idx, w, 2), lambda: moe.moe_route_scored(h, None, idx, w, 2),
                 lambda: moe.moe_route_scored_bwd(x, idx, w[:3], x.clone()),
                 lambda: moe.moe_linear_fwd(x, torch.zeros(64, 60, device="cuda"), None, torch.zeros(4, 60, device="cuda")),
                 lambda: moe.moe_linear_fwd(x, torch.zeros(32, 64, device="cuda"), None, x.clone()),
                 lambda: moe.moe_linear_fwd(h, torch.zeros(64, 64, device="cuda"), None, h.clone()),
                 lambda: moe.moe_linear_fwd(x, torch.zeros(64, 64, device="cuda"), None, x, act=7)):
        with pytest.raises(moe.MoeError):
            call()
