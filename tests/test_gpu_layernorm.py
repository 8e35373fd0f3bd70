"""GPU parity of the layer norm, forward and backward, against the 64-bit
reference of block_ref.py, with bounds counted from the formulas."""
import numpy as np
import pytest
import torch

import block_ref as R
from expert_grouped_gemm_top_amd import moe
from moe_cases import note

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24  # half an fp32 step


def inputs(T, H, dtype, seed, shift=0.3):
    rng = np.random.default_rng(seed)
    r = lambda *s: R.rounded(rng.standard_normal(s), dtype)  # noqa: E731
    return dict(x=R.rounded(rng.standard_normal((T, H)) * 2 + shift, dtype), gamma=R.rounded(1 + 0.3 * rng.standard_normal(H), dtype),
                beta=r(H), dy=r(T, H), dx_add=r(T, H))


def terms(H):
    """Roundings of a row's sum: its adds in a lane (H / 64 at most, or 8 per run), in the wave and over the waves, and the quotient."""
    return max(8, H // 64) + 6 + 4 + 2


def forward(v, dtype, beta=True, eps=1e-5, in_place=False):
    T, H = v["x"].shape
    x = R.dev(v["x"], dtype)
    y = x if in_place else torch.full_like(x, 7.0)
    mean, rstd = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    moe.moe_layernorm_fwd(x, R.dev(v["gamma"], dtype), R.dev(v["beta"], dtype) if beta else None, y, mean, rstd, eps)
    torch.cuda.synchronize()
    return R.host(y), R.host(mean), R.host(rstd)


def check_forward(v, dtype, beta=True, eps=1e-5, in_place=False):
    H = v["x"].shape[1]
    y, mean, rstd = forward(v, dtype, beta, eps, in_place)
    ry, rm, rr = R.norm(v["x"], v["gamma"], v["beta"] if beta else None, eps)
    n = terms(H)
    size = np.abs(v["x"]).mean(1)           # of the terms of the mean
    dm = n * STEP * size + STEP * np.abs(rm)
    R.within("mean", mean, rm, dm)
    # the variance: n roundings, and twice the mean's error times the mean difference (0) plus its square
    dv = (n + 3) * STEP + dm * dm * rr * rr
    R.within("rstd", rstd, rr, rr * (dv + 4 * STEP))
    xh = np.abs(v["x"] - rm[:, None]) * rr[:, None]
    off = np.abs(v["gamma"]) * (rr[:, None] * (dm[:, None] + STEP * np.abs(v["x"])) + xh * (dv + 8 * STEP)[:, None])
    R.within("y", y, ry, R.U[dtype] * np.abs(ry) + 1.01 * off + 2 * STEP * (np.abs(ry) + np.abs(v["beta"])))


WIDTHS = [8, 64, 200, 512, 520, 1024, 1032, 1536, 2048, 2880, 4096, 4104, 8192, 8200, 16384]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward(H, dtype):
    for T in (1, 2, 5, 67):
        note(f"norm T={T} H={H} {dtype}")
        check_forward(inputs(T, H, dtype, T + H), dtype, beta=T != 2, in_place=T == 5)


def test_forward_of_shifted_and_constant_rows():
    """Means far above the spread, where a sum of squares would lose the variance; rows without a spread."""
    for dtype in ("f32", "bf16"):
        v = inputs(9, 2048, dtype, 3, shift=1000.0)
        v["x"][4] = 5.0
        v["x"][5] = 0.0
        check_forward(v, dtype)


def test_forward_nan_and_infinite_rows_stay_in_their_row():
    v = inputs(6, 1032, "bf16", 4)
    v["x"][1, 700], v["x"][3, 5] = np.nan, np.inf
    y, mean, rstd = forward(v, "bf16")
    ok = [0, 2, 4, 5]
    assert np.isnan(y[[1, 3]]).all() and np.isfinite(y[ok]).all()
    ref = R.norm(v["x"][ok], v["gamma"], v["beta"], 1e-5)[0]
    assert np.abs(y[ok] - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-4


def backward(v, dtype, beta=True, add=False, alias=None):
    T, H = v["x"].shape
    _, m, r = R.norm(v["x"], v["gamma"], None, 1e-5)
    m32, r32 = np.float32(m), np.float32(r)
    t = {n: R.dev(v[n], dtype) for n in ("x", "gamma", "dy", "dx_add")}
    dx = t[alias] if alias else torch.full_like(t["x"], 7.0)
    dga, dbe = torch.full_like(t["gamma"], 7.0), torch.full_like(t["gamma"], 7.0)
    need = moe.moe_layernorm_workspace_bytes(T, H)
    ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    moe.moe_layernorm_bwd(t["x"], t["gamma"], torch.from_numpy(m32).cuda(), torch.from_numpy(r32).cuda(), t["dy"], dx,
                          dga, dbe if beta else None, ws[:need], t["dx_add"] if add else None)
    torch.cuda.synchronize()
    assert (ws[need:] == 0xAB).all(), "written past the workspace"
    return (R.host(dx), R.host(dga), R.host(dbe)), (m32.astype(np.float64), r32.astype(np.float64))


def check_backward(v, dtype, **how):
    T, H = v["x"].shape
    (dx, dga, dbe), (m, r) = backward(v, dtype, **how)
    add = v["dx_add"] if how.get("add") else 0
    rx, rg, rb = R.norm_bwd(v["x"], v["gamma"], m, r, v["dy"], add)
    n = terms(H) + 8
    xh = np.abs(v["x"] - m[:, None]) * r[:, None]
    dxh = 4 * STEP * (xh + r[:, None] * np.abs(v["x"]))  # the difference and the product
    g = np.abs(v["dy"] * v["gamma"])
    off = r[:, None] * (6 * STEP * g + n * STEP * g.mean(1, keepdims=True) + xh * n * STEP * (g * xh).mean(1, keepdims=True)
                        + dxh * (g * xh).mean(1, keepdims=True) + xh * (g * dxh).mean(1, keepdims=True))
    R.within("dx", dx, rx, R.U[dtype] * np.abs(rx) + 1.01 * off + 2 * STEP * np.abs(add))
    N = T + 8
    R.within("dgamma", dga, rg, R.U[dtype] * np.abs(rg) + 1.01 * ((N * STEP * np.abs(v["dy"]) * xh).sum(0)
                                                                + (np.abs(v["dy"]) * dxh).sum(0)))
    if how.get("beta", True):
        R.within("dbeta", dbe, rb, R.U[dtype] * np.abs(rb) + 1.01 * (N * STEP * np.abs(v["dy"])).sum(0))
    else:
        assert (dbe == 7.0).all()


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward(H, dtype):
    for T in (1, 3, 70):
        note(f"norm bwd T={T} H={H} {dtype}")
        check_backward(inputs(T, H, dtype, T + H), dtype, beta=T != 3, add=T == 3)


@pytest.mark.parametrize("alias", ["x", "dy", "dx_add"])
def test_backward_in_place(alias):
    for H in (256, 2048, 4104):
        note(f"norm bwd in place of {alias} H={H}")
        check_backward(inputs(50, H, "bf16", 8), "bf16", add=True, alias=alias)


def test_backward_of_many_rows():
    for T, H, dtype in ((4099, 64, "bf16"), (5000, 2048, "bf16"), (2100, 1000, "f32")):
        note(f"norm bwd T={T} H={H} {dtype}")
        check_backward(inputs(T, H, dtype, 9), dtype, add=True)


def test_rows_behind_the_last_are_left():
    x = torch.ones(12, 256, device="cuda")
    y = torch.full((12, 256), 7.0, device="cuda")
    gamma = torch.ones(256, device="cuda")
    moe.moe_layernorm_fwd(x[:9], gamma, None, y[:9])
    torch.cuda.synchronize()
    assert (y[9:] == 7.0).all() and (y[:9] == 0.0).all()


def test_more_rows_than_one_grid_row():
    """2^26 narrow rows and some: more than 2^32 threads.  All rows but the last are zeros, whose norm is beta."""
    T, H, n = (1 << 26) + 701, 8, 300
    note(f"norm T={T} H={H}")
    v = inputs(n, H, "bf16", 12)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[-n:] = R.dev(v["x"], "bf16")
    y, mean, rstd = torch.full_like(x, 7.0), torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    gamma, beta = R.dev(v["gamma"], "bf16"), R.dev(v["beta"], "bf16")
    moe.moe_layernorm_fwd(x, gamma, beta, y, mean, rstd)
    torch.cuda.synchronize()
    ry, _, _ = R.norm(v["x"], v["gamma"], v["beta"], 1e-5)
    # as in test_rows_past_32_bits, with the values' own size (a row of 8 is at most sqrt(8) deviations from its mean)
    R.within("y", R.host(y[-n:]), ry, 2.0 ** -8 * np.abs(ry) + 200 * 30 * STEP)
    assert (y[:-n] == beta).all() and (mean[:-n] == 0).all() and (rstd[:-n] == rstd[0]).all()


def test_rows_past_32_bits():
    """More than 2^31 elements: the last rows forward and backward, and dgamma over all."""
    T, H = (1 << 31) // 4096 + 700, 4096
    note(f"norm T={T} H={H}")
    v = inputs(300, H, "bf16", 11)
    x, dy = torch.ones(T, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[-300:], dy[-300:] = R.dev(v["x"], "bf16"), R.dev(v["dy"], "bf16")
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    gamma, beta = R.dev(v["gamma"], "bf16"), R.dev(v["beta"], "bf16")
    moe.moe_layernorm_fwd(x, gamma, beta, y, mean, rstd)
    dga, dbe = torch.empty_like(gamma), torch.empty_like(gamma)
    ws = torch.empty(moe.moe_layernorm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    last = R.host(y[-300:])
    moe.moe_layernorm_bwd(x, gamma, mean, rstd, dy, y, dga, dbe, ws)
    torch.cuda.synchronize()
    ry, rm, rr = R.norm(v["x"], v["gamma"], v["beta"], 1e-5)
    # half a bf16 step and what check_forward counts for fp32, here at most 200 half steps of values below 30
    R.within("y", last, ry, 2.0 ** -8 * np.abs(ry) + 200 * 30 * STEP)
    rx, rg, rb = R.norm_bwd(v["x"], v["gamma"], rm, rr, v["dy"])
    R.within("dx", R.host(y[-300:]), rx, 2.0 ** -8 * np.abs(rx) + 400 * 30 * STEP)
    assert (y[:-300] == 0).all()
    # the other rows add exact zeros; sums of 300 terms below 30
    R.within("dgamma", R.host(dga), rg, 2.0 ** -8 * np.abs(rg) + 320 * 300 * 5 * STEP)
    R.within("dbeta", R.host(dbe), rb, 2.0 ** -8 * np.abs(rb) + 320 * 300 * 5 * STEP)
