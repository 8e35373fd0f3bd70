"""Plain 64-bit references (numpy) of the operators behind the block: the balance
loss, the vocabulary loss and AdamW, with the elementwise bounds their tests hold
the kernels to (block_ref.py has the rules they count by)."""
from __future__ import annotations

import numpy as np

SOFTMAX, SIGMOID = 0, 1
INF = float("inf")

# ---- balance loss ----------------------------------------------------------------


def shares(l, score):
    """Each expert's share, by the formula; rows without an available expert: 0; NaN rows stay NaN."""
    l = np.asarray(l, np.float64)
    with np.errstate(all="ignore"):
        a = l if score == SOFTMAX else -np.logaddexp(0.0, -l)
        top = a.max(1, keepdims=True)
        e = np.exp(a - np.where(top == -INF, 0.0, top))
        total = e.sum(1, keepdims=True)
        return np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))


def sequences(T, offsets):
    """The sequence of every row, -1 for none."""
    seq = np.full(T, -1)
    for s in range(len(offsets) - 1):
        seq[max(0, offsets[s]):max(0, min(T, offsets[s + 1]))] = s
    return seq


def balance(l, idx, offsets, score, alpha):
    T, E = l.shape
    S, k = len(offsets) - 1, idx.shape[1]
    seq, p = sequences(T, offsets), shares(l, score)
    counts, mean = np.zeros((S, E), np.int64), np.zeros((S, E))
    for s in range(S):
        rows = seq == s
        i = idx[rows].reshape(-1)
        counts[s] = np.bincount(i[(i >= 0) & (i < E)], minlength=E)
        if rows.any():
            mean[s] = p[rows].mean(0)
    n = (seq >= 0).sum()
    return counts, mean, alpha * E / k / n * (counts * mean).sum() if n else 0.0


def balance_bwd(l, counts, k, offsets, score, alpha, dloss):
    """dl, and what its rounding errors are counted by: |factor| p (|d_e| + sum_j p_j |d_j|), d the difference to
    the likeliest expert's count."""
    T, E = l.shape
    seq, p = sequences(T, offsets), shares(l, score)
    n_s = np.bincount(seq[seq >= 0], minlength=len(offsets) - 1)
    dl, size = np.zeros((T, E)), np.zeros((T, E))
    if not n_s.sum():
        return dl, size
    with np.errstate(all="ignore"):
        slope = np.ones_like(p) if score == SOFTMAX else np.exp(-np.logaddexp(0.0, np.asarray(l, np.float64)))
    for t in np.flatnonzero(seq >= 0):
        c = counts[seq[t]].astype(np.float64)
        f = dloss * alpha * E / k / n_s.sum() / n_s[seq[t]]
        d = c - c[np.nanargmax(np.where(np.isnan(l[t]), -INF, l[t]))]
        dl[t] = f * p[t] * slope[t] * (d - (p[t] * d).sum())
        size[t] = abs(f) * p[t] * slope[t] * (np.abs(d) + (p[t] * np.abs(d)).sum())
    return dl, size


# ---- vocabulary loss ---------------------------------------------------------------


def vocab(x, w, y, n_classes, dloss=None, scale=1.0):
    """loss, lse, mean, dx and dw in 64 bits, and what the gradients' errors are counted by: the sums of their terms'
    sizes.  Rows that are not counted are not looked at."""
    T, V = len(y), w.shape[1]
    rows = np.flatnonzero((y >= 0) & (y < n_classes))
    n = len(rows)
    loss, lse, dx, dw = np.zeros(T), np.zeros(T), np.zeros(x.shape), np.zeros(w.shape)
    sx, sw = np.zeros(x.shape), np.zeros(w.shape)
    l = x[rows] @ w[:, :n_classes]
    own = l[np.arange(n), y[rows]]
    with np.errstate(all="ignore"):
        others = l.copy()
        others[np.arange(n), y[rows]] = -INF
        top = np.maximum(others.max(1), -1e300) if n else np.zeros(0)
        d = top + np.log(np.exp(others - top[:, None]).sum(1)) - own
        loss[rows] = np.logaddexp(0.0, d)
    lse[rows] = own + loss[rows]
    p = np.exp(l - lse[rows][:, None])
    p[np.arange(n), y[rows]] = np.expm1(-loss[rows])
    c = scale * (1.0 / max(n, 1) if dloss is None else 1.0)
    p = p * (1.0 if dloss is None else dloss[rows][:, None]) * c
    dx[rows] = p @ w[:, :n_classes].T
    dw[:, :n_classes] = x[rows].T @ p
    sx[rows] = np.abs(p) @ np.abs(w[:, :n_classes]).T
    sw[:, :n_classes] = np.abs(x[rows]).T @ np.abs(p)
    mean = np.array([loss.sum() / n, 1.0 / n]) if n else np.zeros(2)
    # the size of a logit's terms, row by row: what rounding its sum is counted by
    size = np.zeros(T)
    if n:
        size[rows] = (np.abs(x[rows]) @ np.abs(w[:, :n_classes])).max(1)
    return dict(loss=loss, lse=lse, mean=mean, dx=dx, dw=dw, sx=sx, sw=sw, size=size, n=n)


# ---- AdamW -----------------------------------------------------------------------


def mix(x):
    x = np.asarray(x, np.uint64)
    M = np.uint64(0xffffffff)
    x = (x ^ (x >> np.uint64(16))) * np.uint64(0x85ebca77) & M
    x = (x ^ (x >> np.uint64(15))) * np.uint64(0xc2b2ae3d) & M
    return x ^ (x >> np.uint64(16))


def dither(first_block, n, step, seed):
    """32 bits for each element of a tensor whose first block has that number."""
    place = np.arange(n, dtype=np.uint64) + np.uint64(256 * first_block)
    key = mix((mix(step) + np.uint64(seed)) & np.uint64(0xffffffff))
    return mix(place ^ key)


M_VALUES = np.array([c * 2.0 ** -9 if c < 8 else (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7) for c in range(127)])
V_VALUES = np.array([0.0] + [(8 + c % 8) * 2.0 ** (c // 8 - 34) for c in range(1, 255)])


def values(codes, scale, which):
    table = M_VALUES if which == "m" else V_VALUES
    c = codes.astype(np.int64)
    sign = np.where(c >= 128, -1.0, 1.0) if which == "m" else 1.0
    c = c & 127 if which == "m" else c
    ok = c < len(table)
    v = np.where(ok, table[np.where(ok, c, 0)], np.nan) * sign
    return v * np.repeat(np.asarray(scale, np.float64), 256)[:len(c)]


def codes(a, which, share):
    """Codes and scales of a in 64 bits: the neighbour below, or the one above where what is left over of the gap and
    `share` add up to 1."""
    table, most = (M_VALUES, 448.0) if which == "m" else (V_VALUES, 1.75)
    n, nb = len(a), -(-len(a) // 256)
    size = np.zeros(nb * 256)
    fine = np.isfinite(a)
    with np.errstate(over="ignore"):
        size[:n] = np.where(fine, np.minimum(np.abs(a).astype(np.float32), np.finfo(np.float32).max), 0.0)
    top = size.reshape(nb, 256).max(1)
    e = np.where(top > 0, np.ceil(np.log2(np.where(top > 0, top, 1.0) / most)), -126).astype(int)
    e = np.where(most * 2.0 ** (e - 1.0) >= top, e - 1, e)
    e = np.where(most * 2.0 ** e.astype(float) < top, e + 1, e)
    scale = 2.0 ** np.clip(e, -126, 127).astype(float)
    x = np.where(fine, np.abs(a), 0.0) / np.repeat(scale, 256)[:n]
    at = np.minimum(np.searchsorted(table, x, side="right") - 1, len(table) - 1)
    up = np.minimum(at + 1, len(table) - 1)
    gap = np.where(up > at, table[up] - table[at], 1.0)
    c = np.where((x - table[at]) / gap + share >= 1.0, up, at)
    if which == "v":
        c = np.where((at == 0) & (x > 0), 1, c)
        return np.where(fine, c, 255).astype(np.uint8), scale.astype(np.float32)
    c = np.where(fine, c, 127)
    return (c + 128 * ((a < 0) & fine)).astype(np.uint8), scale.astype(np.float32)


def adamw(p, g, m, v, step, lr, b1, b2, eps, decay, gs):
    """The step in 64 bits, and the error that fp32 arithmetic may leave in p: 2^-24 of p for each of three roundings,
    of the update for sixteen, and what m's four leave where its two terms cancel."""
    g = g * gs
    m1 = b1 * m + (1 - b1) * g
    v1 = b2 * v + (1 - b2) * g * g
    c1, c2 = 1 - b1 ** step, 1 - b2 ** step
    den = np.sqrt(v1 / c2) + eps
    with np.errstate(all="ignore"):
        upd = lr * (m1 / c1) / den
        slack = lr / c1 / den * (np.abs(b1 * m) + np.abs((1 - b1) * g))
    p1 = p * (1 - lr * decay) - upd
    return p1, m1, v1, 2.0 ** -24 * (3 * np.abs(p) + 16 * np.abs(upd) + 4 * slack)
