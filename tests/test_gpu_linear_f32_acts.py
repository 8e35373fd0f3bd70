"""The fp32 linear product's activations and slopes, relative to their own size
(the bounds of test_gpu_linear.py allow an absolute error next to 0): values far
into the tails, given exactly as pre-activations.

Half steps (2^-24) counted for fp32: expf 6, erfcf 32, a division 5, one each
for a constant, a product, a sum.  s = logistic(v) from exp(-|v|) has 12 and its
argument's error times |v|; 1 - s formed as logistic(-v) the same."""
import math

import numpy as np
import pytest
import torch

import block_ref as R
from expert_grouped_gemm_top_amd import moe
from moe_cases import note

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24
A, B = math.sqrt(2 / math.pi), 0.044715


def points():
    z = np.concatenate([np.linspace(-12, 12, 481), np.linspace(-86, 86, 173), [-0.75179, 1e-20, -1e-20, 0.0, -3.0, -2.0],
                        np.geomspace(1e-6, 1e-1, 20), -np.geomspace(1e-6, 1e-1, 20)])
    z = np.float32(np.concatenate([z, np.zeros(-len(z) % 8)]))
    return z.astype(np.float64)


def cdf(z):
    return 0.5 * torch.special.erfc(torch.from_numpy(-z * math.sqrt(0.5))).numpy()


def logistic(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1 + e)


def value(act, z):
    """The activation and its bound in half steps of itself."""
    if act == R.NONE:
        return z, 0 * z
    if act == R.RELU:
        return np.maximum(z, 0), 0 * z
    if act == R.SILU:
        return z * logistic(z), 0 * z + 14
    if act == R.GELU:  # the argument's 2 half steps times erfc's condition, at most z^2 + 1
        return z * cdf(z), 2 * (z * z + 1) + 34
    u = 2 * A * (z + B * z ** 3)
    return z * logistic(u), 7 * np.abs(u) + 14


def slope(act, z):
    """The slope and its absolute bound: of each of its terms, and one half step of the sum."""
    if act == R.NONE:
        return np.ones_like(z), 0 * z
    if act == R.RELU:
        return (z > 0) * 1.0, 0 * z
    if act == R.SILU:
        s, c = logistic(z), logistic(-z)
        return s * (1 + z * c), HALF * (12 + 12 + 8) * s * (1 + np.abs(z) * c)
    if act == R.GELU:
        p, t = cdf(z), z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return p + t, HALF * ((2 * (z * z + 1) + 34) * p + (z * z + 12) * np.abs(t))
    u = 2 * A * (z + B * z ** 3)
    s, t = logistic(u), z * logistic(u) * logistic(-u) * 2 * A * (1 + 3 * B * z * z)
    return s + t, HALF * ((7 * np.abs(u) + 14) * s + (14 * np.abs(u) + 36) * np.abs(t))


@pytest.mark.parametrize("act", range(5))
def test_values(act):
    """One row of x picks the first row of w: z is that row exactly."""
    note(f"fp32 activation {act}")
    z = points()
    w = np.zeros((8, len(z)))
    w[0] = z
    x = np.zeros((3, 8))
    x[:, 0] = 1.0
    y, zs = (torch.full((3, len(z)), 7.0, device="cuda") for _ in range(2))
    ws = torch.empty(moe.moe_linear_workspace_bytes(3, 8, len(z), torch.float32) + 16, dtype=torch.uint8, device="cuda")
    moe.moe_linear_fwd(R.dev(x, "f32"), R.dev(w, "f32"), None, y, act, z_save=zs, workspace=ws)
    torch.cuda.synchronize()
    ref, n = value(act, z)
    for t in range(3):
        assert np.array_equal(R.host(zs)[t], z)
        # a factor below 2^-126 may be cut off
        R.within("y", R.host(y)[t], ref, 1.01 * n * HALF * np.abs(ref) + (np.abs(z) + 1) * 2.0 ** -126)


@pytest.mark.parametrize("act", range(5))
def test_slopes_and_values_of_the_backward(act):
    """With dy = mul = 1, dz is the slope and dmul the value."""
    note(f"fp32 slope {act}")
    z = points()
    one = torch.ones(2, len(z), device="cuda")
    zd = R.dev(np.tile(z, (2, 1)), "f32")
    dz, dm, dw = torch.full_like(one, 7.0), torch.full_like(one, 7.0), torch.empty(8, len(z), device="cuda")
    ws = torch.empty(moe.moe_linear_workspace_bytes(2, 8, len(z), torch.float32) + 16, dtype=torch.uint8, device="cuda")
    moe.moe_linear_bwd(torch.zeros(2, 8, device="cuda"), torch.zeros(8, len(z), device="cuda"), one, dz, None, dw,
                       act=act, z=zd, mul=torch.ones_like(one), dmul=dm, workspace=ws)
    torch.cuda.synchronize()
    ref, n = value(act, z)
    slo, bound = slope(act, z)
    small = (np.abs(z) + 1) * 2.0 ** -126
    for t in range(2):
        R.within("dmul", R.host(dm)[t], ref, 1.01 * n * HALF * np.abs(ref) + small)
        R.within("dz", R.host(dz)[t], slo, 1.01 * bound + small * (1 + z * z))


@pytest.mark.parametrize("act", range(1, 5))
def test_far_out(act):
    """Pre-activations from 200 in size to the largest: values z and 0, slopes 1 and 0, to the last bit (what is
    left of them is below exp(-200), far below the smallest fp32 number, also times the largest)."""
    note(f"fp32 activation {act} far out")
    top = float(np.finfo(np.float32).max)
    z = np.array([v * s for v in (200.0, 1e4, 1e15, 1e30, 3e38, top, 1e38, 250.0) for s in (1, -1)])
    z = np.float32(z).astype(np.float64)
    n = len(z)
    ws = torch.empty(moe.moe_linear_workspace_bytes(2, 8, n, torch.float32), dtype=torch.uint8, device="cuda")
    x, w = np.zeros((2, 8)), np.zeros((8, n))
    x[:, 0], w[0] = 1.0, z
    y = torch.full((2, n), 7.0, device="cuda")
    moe.moe_linear_fwd(R.dev(x, "f32"), R.dev(w, "f32"), None, y, act, workspace=ws)
    one = torch.ones(2, n, device="cuda")
    dz, dm = torch.full_like(one, 7.0), torch.full_like(one, 7.0)
    moe.moe_linear_bwd(torch.zeros(2, 8, device="cuda"), torch.zeros(8, n, device="cuda"), one, dz, None, None, act=act,
                       z=R.dev(np.tile(z, (2, 1)), "f32"), mul=one, dmul=dm, workspace=ws)
    torch.cuda.synchronize()
    for t in range(2):
        assert np.array_equal(R.host(y)[t], np.maximum(z, 0)), "y"
        assert np.array_equal(R.host(dm)[t], np.maximum(z, 0)), "dmul"
        assert np.array_equal(R.host(dz)[t], (z > 0) * 1.0), "dz"
