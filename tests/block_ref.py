"""Plain 64-bit references (numpy) of the operators around the expert path:
routing by scores, layer norm and the linear product with its epilogue, each
with its gradient, and the elementwise bounds their tests hold the kernels to.

Bounds: a result stored in a type is off by at most half a step, U[type]
relative to its value; a sum of n fp32 terms is off by at most
n 2^-23 sum|terms| in any order (2^-24 for each rounded addition, and as much
again for matrix-core additions, which need not round to nearest).
"""
from __future__ import annotations

import math

import numpy as np
import torch

U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SOFTMAX, SIGMOID = 0, 1
NONE, RELU, GELU, GELU_TANH, SILU = range(5)
INF = float("inf")


def rounded(a, dtype):
    """The values of `a` as the type holds them, in float64."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float64)).to(DT[dtype]).double().numpy()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, np.float64)).to(DT[dtype]).cuda()


def host(t):
    return t.detach().double().cpu().numpy()


def within(name, got, ref, bound):
    """|got - ref| <= bound elementwise; infinities and NaN where the reference has them."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{name}: NaN in other places"
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), f"{name}: infinities differ"
    off = np.where(fine, np.abs(np.where(fine, got, 0) - np.where(fine, ref, 0)), 0)
    over = off - np.where(fine, np.broadcast_to(bound, off.shape), 0)
    at = np.unravel_index(int(np.argmax(over)), over.shape)
    assert over[at] <= 0, f"{name}{list(at)}: {got[at]!r} for {ref[at]!r}, off by {off[at]:.3e}, bound " \
                          f"{np.broadcast_to(bound, off.shape)[at]:.3e}"


def mm(a, b):
    """a @ b in float64, on the GPU where it is large."""
    if a.shape[0] * a.shape[1] * b.shape[1] < 1 << 28:
        return a @ b
    return (torch.from_numpy(np.ascontiguousarray(a)).cuda() @ torch.from_numpy(np.ascontiguousarray(b)).cuda()).cpu().numpy()


# ---- routing by scores ----------------------------------------------------------


def scores(l, score):
    l = np.asarray(l, np.float64)
    with np.errstate(all="ignore"):
        if score == SIGMOID:
            return 1.0 / (1.0 + np.exp(-l))
        m = l.max(1, keepdims=True)
        e = np.where(l == -INF, 0.0, np.exp(l - m))
        z = e.sum(1, keepdims=True)
        s = np.where(z == 0, 0.0, e / z)
    bad = np.isnan(l).any(1) | (l == INF).any(1)
    s[bad] = np.nan
    return s


def _ranked(c):
    """Indices of each row by value descending, NaN first, equal values by index."""
    key = np.where(np.isnan(c), INF, c)
    order = np.argsort(-key, axis=1, kind="stable")
    # NaN above +inf: a stable second pass on the NaN flag
    flag = np.take_along_axis(np.isnan(c), order, axis=1)
    return np.take_along_axis(order, np.argsort(~flag, axis=1, kind="stable"), axis=1)


def route(l, bias, k, score, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    l = np.asarray(l, np.float64)
    T, E = l.shape
    s = scores(l, score)
    gone = l == -INF
    c = np.where(gone, -INF, s + (0.0 if bias is None else np.asarray(bias, np.float64)))
    rank_by = c if bias is not None else l.copy()
    if groups > 1:
        size = E // groups
        if group_top == 1:
            v = rank_by.reshape(T, groups, size)
            worth = np.where(np.isnan(v).any(2), np.nan, v.max(2))
        else:
            v = c.reshape(T, groups, size)
            two = -np.sort(-v, axis=2)[:, :, :2]
            worth = np.where(two[:, :, 1] == -INF, two[:, :, 0], two.sum(2))
            worth = np.where(np.isnan(v).any(2), np.nan, worth)
        kept = np.zeros((T, groups), bool)
        np.put_along_axis(kept, _ranked(worth)[:, :top_groups], True, axis=1)
        rank_by = np.where(np.repeat(kept, size, axis=1), rank_by, -INF)
    idx = _ranked(rank_by)[:, :k]
    return idx.astype(np.int32), weights(l, idx, score, renorm, scale)


def undecided(l, bias, k, score, groups=1, top_groups=1, group_top=1):
    """Tokens whose choice 64-bit arithmetic does not define: two different sums (a choice score s + b, or the
    worth of a group) next to the border that are equal as real numbers, or as good as.  A sum of up to four
    terms below 2 is off by at most 4 ulp, 2^-50, and either side may round the other way: 2^-48 apart decides.
    Sums of the same logits and biases are equal on both sides and go by index."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    c = np.where(l == -INF, -INF, scores(l, score) + b)
    out = np.zeros(T, bool)
    if bias is None and (groups == 1 or group_top == 1):
        return out
    near = 2.0 ** -48
    for t in range(T):
        order = _ranked(c[t:t + 1])[0]
        if groups > 1:
            size = E // groups
            best = [sorted(range(g * size, (g + 1) * size), key=lambda e: -c[t, e])[:group_top] for g in range(groups)]
            worth = np.array([sum(c[t, e] for e in m if c[t, e] > -INF) if c[t, m[0]] > -INF else -INF for m in best])
            by = np.argsort(-worth, kind="stable")
            edge = by[top_groups - 1]
            for g in by:  # any group as good as the last kept one, but from other terms
                same = [(l[t, e], b[e]) for e in best[g]] == [(l[t, e], b[e]) for e in best[edge]]
                if g != edge and abs(worth[g] - worth[edge]) <= near and not same:
                    out[t] = True
            kept = set(by[:top_groups])
            order = [e for e in order if e // size in kept]
        if bias is not None:
            for i, j in zip(order[:k], order[1:k + 1]):
                if abs(c[t, i] - c[t, j]) <= near and (l[t, i], b[i]) != (l[t, j], b[j]):
                    out[t] = True
    return out


def weights(l, idx, score, renorm, scale):
    """Of the selected experts, from log scores: ratios that do not underflow."""
    l = np.asarray(l, np.float64)
    s = np.take_along_axis(scores(l, score), idx, axis=1)
    if not renorm:
        return scale * s
    sel = np.take_along_axis(l, idx, axis=1)
    with np.errstate(all="ignore"):
        a = sel if score == SOFTMAX else -np.logaddexp(0.0, -sel)
        a = np.where(sel == -INF, -INF, a)
        m = a.max(1, keepdims=True)
        e = np.where(a == -INF, 0.0, np.exp(a - np.where(m == -INF, 0.0, m)))
        z = e.sum(1, keepdims=True)
        p = np.where(z == 0, 0.0, e / z)
    p[np.isnan(s).any(1)] = np.nan
    return scale * p


def route_bwd(l, idx, g, score, renorm, scale):
    l, g = np.asarray(l, np.float64), np.asarray(g, np.float64)
    out = np.zeros_like(l)
    s_all = scores(l, score)
    s = np.take_along_axis(s_all, idx, axis=1)
    if renorm:
        p = weights(l, idx, score, True, 1.0)
        d = scale * p * (g - (p * g).sum(1, keepdims=True))
        d = d if score == SOFTMAX else d * (1 - s)
    elif score == SIGMOID:
        d = scale * g * s * (1 - s)
    else:
        d = scale * s * g
        out -= scale * s_all * (s * g).sum(1, keepdims=True)
    for j in range(idx.shape[1]):
        np.add.at(out, (np.arange(l.shape[0]), idx[:, j]), d[:, j])
    return out


# ---- layer norm -----------------------------------------------------------------


def norm(x, gamma, beta, eps):
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1 / np.sqrt((xc * xc).mean(1) + eps)
    return xc * rstd[:, None] * gamma + (0 if beta is None else beta), mean, rstd


def norm_bwd(x, gamma, mean, rstd, dy, dx_add=None):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx + (0 if dx_add is None else dx_add), (dy * xh).sum(0), dy.sum(0)


# ---- linear ---------------------------------------------------------------------


def _erf(v):
    return torch.erf(torch.from_numpy(np.ascontiguousarray(v))).numpy()


def act(a, z):
    if a == RELU:
        return np.where(z < 0, 0.0, z)
    if a == GELU:
        return 0.5 * z * (1 + _erf(z * math.sqrt(0.5)))
    if a == GELU_TANH:
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if a == SILU:
        with np.errstate(over="ignore"):
            return z / (1 + np.exp(-z))
    return z


def slope(a, z):
    if a == RELU:
        return (z > 0).astype(np.float64)
    if a == GELU:
        return 0.5 * (1 + _erf(z * math.sqrt(0.5))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if a == GELU_TANH:
        t = np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if a == SILU:
        with np.errstate(over="ignore"):
            s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def linear(x, w, bias, a, mul=None, residual=None):
    z = mm(x, w) + (0 if bias is None else bias)
    y = act(a, z) * (1 if mul is None else mul)
    return y + (0 if residual is None else residual), z


def linear_dz(z, mul, dy, a):
    dz = dy * (1 if mul is None else mul)
    if a != NONE:
        dz = dz * slope(a, z)
    return dz, None if mul is None else dy * act(a, z)
