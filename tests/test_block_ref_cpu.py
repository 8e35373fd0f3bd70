"""The 64-bit references of the operators around the expert path against
differences, autograd and hand-made cases: what the GPU tests compare with."""
import numpy as np
import pytest
import torch

import block_ref as R

INF = float("inf")


def differences(f, x, h):
    """Central differences of the scalar f at every entry of x."""
    out = np.zeros_like(x)
    for at in np.ndindex(x.shape):
        lo, hi = x.copy(), x.copy()
        lo[at] -= h
        hi[at] += h
        out[at] = (f(hi) - f(lo)) / (2 * h)
    return out


# central differences with h = 1e-5: truncation h^2 |f'''| / 6 and cancellation 2^-52 |f| / h, both below 1e-8 here
TOL = 1e-7


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    l = rng.standard_normal((3, 7))
    g = rng.standard_normal((3, 4))
    idx, _ = R.route(l, None, 4, score, renorm=renorm, scale=1.7)
    f = lambda v: float((R.weights(v, idx, score, renorm, 1.7) * g).sum())  # noqa: E731
    assert np.abs(R.route_bwd(l, idx, g, score, renorm, 1.7) - differences(f, l, 1e-5)).max() < TOL


def test_route_rules_by_hand():
    l = np.array([[0.0, 1.0, 1.0, -INF, 2.0, 0.5]])
    assert R.route(l, None, 6, R.SIGMOID)[0].tolist() == [[4, 1, 2, 5, 0, 3]]
    # a bias moves the choice, not the weight; an unavailable expert stays out of reach of its bias
    idx, w = R.route(l, [0, 0, 0.1, 9, 0, 9], 2, R.SIGMOID, renorm=False)
    # (0.881 for expert 4, 0.831 for expert 2)
    assert idx.tolist() == [[5, 4]] and np.allclose(w, 1 / (1 + np.exp([[-0.5, -2.0]])))
    # groups of two: worth by the best one, or by both
    assert R.route(l, None, 2, R.SIGMOID, 3, 1, 1)[0].tolist() == [[4, 5]]
    l = np.array([[3.0, -3.0, 1.0, 2.0, 0.0, 0.0]])
    assert R.route(l, None, 2, R.SIGMOID, 3, 1, 1)[0].tolist() == [[0, 1]]
    assert R.route(l, None, 2, R.SIGMOID, 3, 1, 2)[0].tolist() == [[3, 2]]
    # nothing available: the first experts, weight 0
    idx, w = R.route(np.full((1, 4), -INF), [1, 2, 3, 4], 2, R.SOFTMAX)
    assert idx.tolist() == [[0, 1]] and not w.any()
    assert R.route(np.array([[1.0, np.nan, INF]]), None, 3, R.SIGMOID)[0].tolist() == [[1, 2, 0]]


def test_norm_gradient_against_autograd_and_differences():
    rng = np.random.default_rng(4)
    x, dy = rng.standard_normal((3, 8)) + 0.5, rng.standard_normal((3, 8))
    gamma, beta = rng.standard_normal(8), rng.standard_normal(8)
    y, mean, rstd = R.norm(x, gamma, beta, 1e-5)
    t = [torch.from_numpy(a).requires_grad_() for a in (x, gamma, beta)]
    out = torch.nn.functional.layer_norm(t[0], (8,), t[1], t[2], 1e-5)
    assert np.abs(out.detach().numpy() - y).max() < 1e-12
    got = R.norm_bwd(x, gamma, mean, rstd, dy)
    for a, b in zip(got, torch.autograd.grad(out, t, torch.from_numpy(dy))):
        assert np.abs(a - b.numpy()).max() < 1e-12
    f = lambda v: float((R.norm(v, gamma, beta, 1e-5)[0] * dy).sum())  # noqa: E731
    assert np.abs(got[0] - differences(f, x, 1e-5)).max() < TOL


@pytest.mark.parametrize("a", range(5))
def test_activation_slopes_against_differences(a):
    z = np.concatenate([np.linspace(-6, 6, 41) + 0.013, [-40.0, 40.0]])
    h = 1e-5
    assert np.abs(R.slope(a, z) - (R.act(a, z + h) - R.act(a, z - h)) / (2 * h)).max() < TOL


def test_linear_gradient_against_differences():
    rng = np.random.default_rng(5)
    x, w = rng.standard_normal((3, 4)), rng.standard_normal((4, 5))
    b, mul, dy = rng.standard_normal(5), rng.standard_normal((3, 5)), rng.standard_normal((3, 5))
    _, z = R.linear(x, w, b, R.SILU, mul)
    dz, dmul = R.linear_dz(z, mul, dy, R.SILU)
    at = dict(x=x, w=w, b=b, mul=mul)
    f = lambda **v: float((R.linear(**{"a": R.SILU, "bias": {**at, **v}["b"],  # noqa: E731
                                       **{n: t for n, t in {**at, **v}.items() if n != "b"}})[0] * dy).sum())
    for name, got in (("x", dz @ w.T), ("w", x.T @ dz), ("b", dz.sum(0)), ("mul", dmul)):
        assert np.abs(got - differences(lambda v: f(**{name: v}), at[name], 1e-5)).max() < TOL, name
