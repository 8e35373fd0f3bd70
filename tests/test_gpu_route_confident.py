"""Gradients of confident routers (moe_route_scored_bwd): scores so near 0 or 1,
or weights so near 1, that forming 1 - s or g - sum p g from rounded values
would lose the result.  The references form the small differences themselves,
and the bounds are relative to the sizes of the terms of
  renormalised:  scale p_j sum_i p_i (g_j - g_i)  [sigmoid: times 1 - s_j]
  sigmoid:       scale g_j s_j (1 - s_j)
  softmax:       scale s_e (sum over the others of s_i (g_e - g_i)),  g = 0 where not selected."""
import numpy as np
import pytest
import torch

import block_ref as R
from expert_grouped_gemm_top_amd import moe
from moe_cases import note

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24  # half an fp32 step


def softmax(l):
    e = np.exp(l - l.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def reference(l, idx, g, score, renorm, scale):
    """The gradient, and the sizes of the terms it is summed from; no index is listed twice."""
    rows = np.arange(len(l))[:, None]
    if score == R.SIGMOID:
        s, rest = 1 / (1 + np.exp(-l)), 1 / (1 + np.exp(l))  # rest = 1 - s
    if renorm:
        a = l[rows, idx] if score == R.SOFTMAX else -np.logaddexp(0.0, -l[rows, idx])
        p = softmax(a)
        apart = g[:, :, None] - g[:, None, :]
        c = 1.0 if score == R.SOFTMAX else rest[rows, idx]
        d, size = (scale * p * c * (p[:, None, :] * v).sum(2) for v in (apart, np.abs(apart)))
    elif score == R.SIGMOID:
        d = scale * g * s[rows, idx] * rest[rows, idx]
        size = d
    else:
        s, full = softmax(l), np.zeros_like(l)
        full[rows, idx] = g
        apart = full[:, :, None] - full[:, None, :]
        return scale * s * (s[:, None, :] * apart).sum(2), abs(scale) * s * (s[:, None, :] * np.abs(apart)).sum(2)
    out, sizes = np.zeros_like(l), np.zeros_like(l)
    out[rows, idx], sizes[rows, idx] = d, np.abs(size)
    return out, sizes


def steps(l, k, score, renorm):
    """Half steps of the product of terms.  expf 6, a division 5, one each for a sum, a product, a difference.
    A renormalised weight: the log score (at most 8 of its own, which is at most |l|max + 1), the difference to the
    largest (1 of it), expf, the sum of k, the quotient.  A plain softmax's score: the exponent's argument and result
    1.5 |d| + 2 for the distance d of the logit from the largest, twice (in the score and in the sum), the sum of E,
    the quotient.  Both stand twice in a product, and sums of k (E) of those follow."""
    top = np.abs(l).max(1, keepdims=True)
    if renorm:
        weight = 9 * (top + 1) + 6 + k + 5
        return 2 * weight + 12 + (k + 8)
    if score == R.SIGMOID:
        return np.full_like(top, 2 * 12 + 4)
    weight = 2 * (1.5 * 2 * top + 2) + l.shape[1] + 5
    return 2 * weight + (l.shape[1] + 8)


def check(l, idx, g, score, renorm, scale):
    T, E = l.shape
    k = idx.shape[1]
    note(f"confident route bwd T={T} E={E} k={k} score={score} renorm={renorm}")
    l, g = np.float32(l), np.float32(g)
    d = torch.full((T, E), 7.0, device="cuda")
    moe.moe_route_scored_bwd(torch.from_numpy(l).cuda(), torch.from_numpy(np.int32(idx)).cuda(),
                             torch.from_numpy(g).cuda(), d, score, renorm, scale)
    torch.cuda.synchronize()
    l, g = l.astype(np.float64), g.astype(np.float64)
    ref, size = reference(l, idx, g, score, renorm, scale)
    # fp32 holds no normal numbers below 2^-126: each factor may be cut off there
    floor = 4 * abs(scale) * (np.abs(g).max() + 1) * 2.0 ** -126
    R.within("dlogits", R.host(d), ref, 1.01 * steps(l, k, score, renorm) * HALF * size + floor)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(128, 8), (256, 16), (20, 3), (7, 2), (3, 3)])
def test_confident_scores(score, renorm, E, k):
    """Selected logits of 8 to 40, where 1 - s of a sigmoid is 3e-4 to 4e-18; the other logits ordinary ones."""
    rng = np.random.default_rng(E + k)
    T = 60
    l = rng.standard_normal((T, E))
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    rows = np.arange(T)[:, None]
    l[rows, idx] = rng.uniform(8, 40, (T, k))
    l[:10] *= -1  # and of -8 to -40
    check(l, idx, rng.standard_normal((T, k)), score, renorm, 2.5)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(128, 8), (64, 4), (37, 5), (2, 2)])
def test_one_weight_near_one(score, renorm, E, k):
    """One selected expert far above all others: its weight is 1 - 1e-3 down to 1 - 1e-17."""
    rng = np.random.default_rng(100 + E)
    T = 60
    l = rng.standard_normal((T, E)) - (6.0 if score == R.SIGMOID else 0.0)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    far = np.linspace(7, 40, T)
    if score == R.SIGMOID:  # the others' scores near 0
        l -= far[:, None]
    l[np.arange(T), idx[:, k // 2]] = far if score == R.SOFTMAX else 1.0
    check(l, idx, rng.standard_normal((T, k)), score, renorm, 1.0)
    check(l, idx, 1.0 + 0.01 * rng.standard_normal((T, k)), score, renorm, -1.5)


@pytest.mark.parametrize("renorm", [False, True])
def test_a_confident_expert_listed_twice(renorm):
    """The two listings' gradients add up; the softmax's expert counts once in the sum over the experts."""
    rng = np.random.default_rng(3)
    T, E, k = 24, 40, 5
    l = rng.standard_normal((T, E))
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    idx[:, 3] = idx[:, 1]
    l[np.arange(T), idx[:, 1]] = np.linspace(6, 30, T)
    g = rng.standard_normal((T, k))
    for score in (R.SOFTMAX, R.SIGMOID):
        note(f"listed twice score={score} renorm={renorm}")
        l32, g32 = np.float32(l), np.float32(g)
        d = torch.full((T, E), 7.0, device="cuda")
        moe.moe_route_scored_bwd(torch.from_numpy(l32).cuda(), torch.from_numpy(np.int32(idx)).cuda(),
                                 torch.from_numpy(g32).cuda(), d, score, renorm, 1.0)
        torch.cuda.synchronize()
        x, y = l32.astype(np.float64), g32.astype(np.float64)
        rows = np.arange(T)[:, None]
        if renorm:  # every listing a term of its own
            a = x[rows, idx] if score == R.SOFTMAX else -np.logaddexp(0.0, -x[rows, idx])
            p = softmax(a)
            apart = y[:, :, None] - y[:, None, :]
            c = 1.0 if score == R.SOFTMAX else 1 / (1 + np.exp(x[rows, idx]))
            ref, size = np.zeros_like(x), np.zeros_like(x)
            for out, v in ((ref, apart), (size, np.abs(apart))):
                np.add.at(out, (rows, idx), p * c * (p[:, None, :] * v).sum(2))
        else:  # as one listing with the sum of both
            once = y.copy()
            once[:, 1] += once[:, 3]
            keep = [0, 1, 2, 4]
            ref, size = reference(x, idx[:, keep], once[:, keep], score, False, 1.0)
            if score == R.SIGMOID:
                two = np.abs(y).copy()
                two[:, 1] += two[:, 3]
                size = np.abs(reference(x, idx[:, keep], two[:, keep], score, False, 1.0)[1])
            else:  # the sum of the two gradients is rounded: a step of its size
                extra = np.zeros_like(x)
                extra[rows, idx[:, 1:2]] = (np.abs(y[:, 1]) + np.abs(y[:, 3]))[:, None]
                s = softmax(x)
                size = size + s * (extra * (1 - s) + (s * extra).sum(1, keepdims=True) * (extra == 0))
        n = steps(x, k, score, renorm) + 4
        R.within("dlogits", R.host(d), ref, 1.01 * n * HALF * size + 32 * 2.0 ** -126)


@pytest.mark.parametrize("score,renorm", [(R.SOFTMAX, True), (R.SIGMOID, True), (R.SIGMOID, False)])
def test_logits_that_are_not_selected_are_not_read(score, renorm):
    """NaN and infinities among them leave the gradient as it is; at a selected one they reach that token."""
    rng = np.random.default_rng(5)
    T, E, k = 20, 48, 4
    l = np.float32(rng.standard_normal((T, E)))
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    g = np.float32(rng.standard_normal((T, k)))
    check(l.astype(np.float64), idx, g, score, renorm, 1.0)
    spoilt = l.copy()
    for t in range(T):
        spoilt[t, np.setdiff1d(np.arange(E), idx[t])[:3]] = np.nan, np.inf, -np.inf
    spoilt[7, idx[7, 2]] = np.nan
    out = []
    for v in (l, spoilt):
        d = torch.full((T, E), 7.0, device="cuda")
        moe.moe_route_scored_bwd(torch.from_numpy(v).cuda(), torch.from_numpy(np.int32(idx)).cuda(),
                                 torch.from_numpy(g).cuda(), d, score, renorm, 1.0)
        torch.cuda.synchronize()
        out.append(R.host(d))
    others = np.arange(T) != 7
    assert np.array_equal(out[0][others], out[1][others])
    bad = np.isnan(out[1][7])
    assert bad[idx[7, 2]] and (bad[idx[7]].all() if renorm else bad.sum() == 1)
    assert not out[1][7, np.setdiff1d(np.arange(E), idx[7])].any()
