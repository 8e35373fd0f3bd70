"""GPU parity of the linear product with its epilogue, forward and backward,
against the 64-bit reference of block_ref.py, with bounds counted from the
formulas: an fp32 sum of n terms is off by at most n 2^-23 of its terms' sizes,
a stored value by half a step, a slope or a value of an activation by its
Lipschitz constant (1.13) times its argument's error and 32 half steps of its own."""
import numpy as np
import pytest
import torch

import block_ref as R
from expert_grouped_gemm_top_amd import moe
from moe_cases import note

pytestmark = pytest.mark.gpu

LIP = 1.13  # the largest slope of the activations (GELU)


def inputs(T, I, O, dtype, seed):  # noqa: E741
    rng = np.random.default_rng(seed)
    r = lambda scale, *s: R.rounded(scale * rng.standard_normal(s), dtype)  # noqa: E731
    return dict(x=r(1, T, I), w=r(I ** -0.5, I, O), b=r(0.5, O), mul=r(1, T, O), residual=r(1, T, O), z=r(1.5, T, O),
                dy=r(1, T, O), dx_add=r(1, T, I))


def workspace(T, I, O, dtype):  # noqa: E741
    need = moe.moe_linear_workspace_bytes(T, I, O, R.DT[dtype])
    return torch.full((need + 64,), 0xAB, dtype=torch.uint8, device="cuda"), need


def check_forward(v, dtype, act, bias=True, mul=False, residual=False, save=True, in_place=None):
    T, I = v["x"].shape  # noqa: E741
    O = v["w"].shape[1]  # noqa: E741
    note(f"linear T={T} I={I} O={O} {dtype} act={act} bias={bias} mul={mul} residual={residual} save={save}")
    t = {n: R.dev(v[n], dtype) for n in ("x", "w", "b", "mul", "residual")}
    y = t[in_place] if in_place else torch.full((T, O), 7.0, dtype=R.DT[dtype], device="cuda")
    z = torch.full((T, O), 7.0, dtype=R.DT[dtype], device="cuda") if save else None
    ws, need = workspace(T, I, O, dtype)
    moe.moe_linear_fwd(t["x"], t["w"], t["b"] if bias else None, y, act, t["mul"] if mul else None,
                       t["residual"] if residual else None, z, ws[:need])
    torch.cuda.synchronize()
    assert (ws[need:] == 0xAB).all(), "written past the workspace"
    m, r = v["mul"] if mul else None, v["residual"] if residual else None
    ry, rz = R.linear(v["x"], v["w"], v["b"] if bias else None, act, m, r)
    dz = (I + 2) * 2.0 ** -23 * (R.mm(np.abs(v["x"]), np.abs(v["w"])) + np.abs(v["b"]))
    if save:
        R.within("z", R.host(z), rz, R.U[dtype] * np.abs(rz) + 1.01 * dz)
    val = np.abs(R.act(act, rz))
    off = (LIP * dz + 32 * 2.0 ** -24 * (val + np.abs(rz) * (act in (R.GELU, R.GELU_TANH)))) * (1 if m is None else np.abs(m))
    if r is not None:
        off = off + 2.0 ** -23 * (np.abs(r) + np.abs(ry))
    R.within("y", R.host(y), ry, R.U[dtype] * np.abs(ry) + 1.01 * off + 2.0 ** -22 * np.abs(ry))


SHAPES = [  # T, I, O: one row, few rows, around tile edges, ragged, long reductions
    (1, 8, 8), (1, 2048, 768), (3, 72, 40), (8, 768, 2048), (15, 256, 136), (16, 512, 512), (17, 40, 264), (33, 1408, 64),
    (64, 64, 64), (65, 200, 136), (127, 136, 200), (130, 2048, 72), (255, 88, 520), (256, 256, 256), (300, 1000, 248),
    (513, 64, 1032), (1000, 776, 264),
]


@pytest.mark.parametrize("T,I,O", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward(T, I, O, dtype):  # noqa: E741
    v = inputs(T, I, O, dtype, T + I + O)
    check_forward(v, dtype, R.NONE, bias=False, save=False)
    check_forward(v, dtype, R.SILU, bias=True, mul=True, residual=True)


LARGE = [  # every workgroup tile with and without masked edges, split reductions, more workgroups than CUs
    (4096, 2048, 4096, "bf16"), (4090, 2040, 4088, "bf16"), (2500, 1024, 2048, "bf16"), (4099, 2048, 768, "bf16"),
    (700, 1032, 1000, "bf16"), (40, 4096, 512, "bf16"), (9, 4104, 4096, "bf16"), (1500, 520, 1032, "f32"),
    (70, 3080, 136, "f32"), (3, 65536, 64, "bf16"), (2, 20000, 40, "f32"),
]


@pytest.mark.parametrize("T,I,O,dtype", LARGE)
def test_forward_large(T, I, O, dtype):  # noqa: E741
    check_forward(inputs(T, I, O, dtype, T + O), dtype, R.GELU_TANH, mul=True, residual=True)


@pytest.mark.parametrize("T,I,O,dtype", LARGE + [
    (4088, 4088, 4080, "bf16"), (8192, 4096, 1408, "bf16"), (8195, 64, 72, "bf16"), (1536, 2048, 4096, "bf16"),
    (1530, 2040, 4088, "bf16"), (1024, 2560, 1000, "bf16"), (1536, 4096, 1408, "bf16"), (1023, 1000, 2048, "bf16")])
def test_backward_large(T, I, O, dtype):  # noqa: E741
    check_backward(inputs(T, I, O, dtype, T + O), dtype, R.SILU, mul=True, add=True)


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,I,O", [(5, 128, 96), (150, 72, 200), (520, 256, 264)])
def test_forward_epilogues(act, dtype, T, I, O):  # noqa: E741
    v = inputs(T, I, O, dtype, act)
    v["x"][0] *= 16.0  # far into the activations' tails
    for bias, mul, residual, save in ((1, 0, 0, 1), (0, 1, 0, 0), (0, 0, 1, 1), (1, 1, 1, 0)):
        check_forward(v, dtype, act, bool(bias), bool(mul), bool(residual), bool(save))


@pytest.mark.parametrize("in_place", ["mul", "residual"])
def test_forward_in_place(in_place):
    for T, I, O in ((4, 64, 96), (200, 128, 264), (600, 264, 520)):  # noqa: E741
        check_forward(inputs(T, I, O, "bf16", 5), "bf16", R.GELU, mul=True, residual=True, in_place=in_place)


def check_backward(v, dtype, act, bias=True, mul=False, add=False, want=("dx", "dw"), dz_in=None, dmul_in=None,
                   add_in_place=False):
    T, I = v["x"].shape  # noqa: E741
    O = v["w"].shape[1]  # noqa: E741
    note(f"linear bwd T={T} I={I} O={O} {dtype} act={act} bias={bias} mul={mul} add={add} want={want}")
    t = {n: R.dev(v[n], dtype) for n in ("x", "w", "z", "mul", "dy", "dx_add")}
    new = lambda *s: torch.full(s, 7.0, dtype=R.DT[dtype], device="cuda")  # noqa: E731
    plain = act == R.NONE and not mul
    dz = None if plain else (t[dz_in] if dz_in else new(T, O))
    dx = (t["dx_add"] if add_in_place else new(T, I)) if "dx" in want else None
    dw = new(I, O) if "dw" in want else None
    db = new(O) if bias else None
    dm = (t[dmul_in] if dmul_in else new(T, O)) if mul else None
    ws, need = workspace(T, I, O, dtype)
    moe.moe_linear_bwd(t["x"], t["w"], t["dy"], dz, dx, dw, db, act, None if plain else t["z"], t["mul"] if mul else None,
                       dm, t["dx_add"] if add and dx is not None else None, ws[:need])
    torch.cuda.synchronize()
    assert (ws[need:] == 0xAB).all(), "written past the workspace"
    m = v["mul"] if mul else None
    rz, rm = R.linear_dz(v["z"], m, v["dy"], act)
    ddz = 40 * 2.0 ** -24 * (np.abs(v["dy"]) * (1 if m is None else np.abs(m)) * (1 + np.abs(v["z"]))) * (not plain)
    stored = (0 if plain else R.U[dtype]) * np.abs(rz) + 1.01 * ddz  # dz as the products read it
    if not plain and dz_in is None:
        R.within("dz", R.host(dz), rz, 1.001 * stored)
    if mul:
        R.within("dmul", R.host(dm), rm, R.U[dtype] * np.abs(rm) * 1.001 + 40 * 2.0 ** -24 * np.abs(v["dy"]) * (1 + np.abs(v["z"])))
    if bias:
        rb = rz.sum(0)
        R.within("dbias", R.host(db), rb, R.U[dtype] * np.abs(rb) * 1.001 + (T + 8) * 2.0 ** -23 * np.abs(rz).sum(0)
                 + ddz.sum(0))
    for name, got, left, right, el, er in (("dx", dx, rz, v["w"].T, stored, 0), ("dw", dw, v["x"].T, rz, 0, stored)):
        if got is None:
            continue
        ref = R.mm(left, right)
        n = left.shape[1]
        size = R.mm(np.abs(left), np.abs(right))
        extra = 0
        if name == "dx" and add:
            ref = ref + v["dx_add"]
            extra = 2.0 ** -23 * (np.abs(v["dx_add"]) + np.abs(ref))
        slip = 0 if plain else (R.mm(el, np.abs(right)) if name == "dx" else R.mm(np.abs(left), er))
        # rounded dz: elementwise at most `slip`; over the whole result the independent roundings (each at
        # most U of its term) add in squares, so the error's norm is at most sqrt(2) U of the result's size
        R.within(name, R.host(got), ref, R.U[dtype] * np.abs(ref) * 1.01 + (n + 2) * 2.0 ** -23 * size + 1.01 * slip + extra)
        if dtype == "bf16" and ref.size > 4096:
            quad = np.sqrt(((left ** 2).sum(0) * (right ** 2).sum(1)).sum() * (not plain) + (ref ** 2).sum())
            assert np.linalg.norm(R.host(got) - ref) <= 1.01 * R.U[dtype] * quad, name


@pytest.mark.parametrize("T,I,O", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward(T, I, O, dtype):  # noqa: E741
    v = inputs(T, I, O, dtype, T + I + O)
    check_backward(v, dtype, R.NONE, bias=True)
    check_backward(v, dtype, R.SILU, bias=False, mul=True, add=True)


@pytest.mark.parametrize("T,I,O", [
    (1, 1024, 1024), (16, 1024, 1024), (33, 1536, 512), (7, 2472, 72), (31, 2000, 200), (5, 4096, 160), (40, 2048, 696),
    (2, 1544, 96), (44, 4096, 64), (16, 512, 4096), (3, 72, 2560), (12, 256, 2048)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_rows(T, I, O, dtype):  # noqa: E741
    """Decoding steps: whole and masked stages of the 32 x 32 tiles, one to several of them, split and not."""
    v = inputs(T, I, O, dtype, T + O)
    check_forward(v, dtype, R.SILU, mul=True, residual=True)
    check_backward(v, dtype, R.SILU, mul=True, add=True)
    check_backward(v, dtype, R.NONE, bias=False, want=("dx",))


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_epilogues(act, dtype):
    v = inputs(150, 72, 200, dtype, act)
    v["z"][0] *= 16.0
    v["z"][1] = 0.0
    for bias, mul, add in ((1, 0, 1), (0, 1, 0), (1, 1, 1), (0, 0, 0)):
        check_backward(v, dtype, act, bool(bias), bool(mul), bool(add))


def test_backward_parts_and_in_place():
    v = inputs(200, 136, 264, "bf16", 6)
    for want in (("dx",), ("dw",), ()):
        check_backward(v, "bf16", R.GELU, want=want)
        check_backward(v, "bf16", R.NONE, want=want)
    check_backward(v, "bf16", R.SILU, mul=True, dz_in="dy", dmul_in="mul", add=True, add_in_place=True)
    check_backward(v, "bf16", R.SILU, mul=True, dz_in="z", dmul_in="dy")


def test_slopes_far_out_are_finite():
    """Pre-activations up to the type's largest value: slopes 0 or 1, no 0 * inf."""
    big = float(torch.finfo(torch.bfloat16).max)
    z = np.tile(np.array([big, -big, 1e4, -1e4, 60.0, -60.0, 0.0, -0.0]), (4, 2))
    v = inputs(4, 8, 16, "bf16", 7)
    v["z"] = R.rounded(z, "bf16")
    t = {n: R.dev(v[n], "bf16") for n in ("x", "w", "z", "dy")}
    for act in range(1, 5):
        note(f"far slopes act={act}")
        dz, dx, dw = torch.empty_like(t["dy"]), torch.empty_like(t["x"]), torch.empty_like(t["w"])
        ws, _ = workspace(4, 8, 16, "bf16")
        moe.moe_linear_bwd(t["x"], t["w"], t["dy"], dz, dx, dw, None, act, t["z"], workspace=ws)
        torch.cuda.synchronize()
        want = np.where(v["z"] > 0, 1.0, 0.0) * v["dy"]
        zero = v["z"] == 0
        want[zero] = 0.0 if act == R.RELU else 0.5 * v["dy"][zero]
        # the slopes are 0 and 1 but for exp(-|z|) times a polynomial in z: at |z| = 60 the SILU's is
        # s (1 + z (1 - s)) with s = exp(-60) (1 - ...), so off 0 or 1 by at most 61 exp(-60) (5.4e-25); the
        # GELUs' tails exp(-z^2 / 2) are smaller still
        R.within("dz", R.host(dz), want, 2.0 ** -8 * np.abs(want) + 62 * np.exp(-60.0) * np.abs(v["dy"]))


def test_nan_stays_in_its_row():
    v = inputs(40, 64, 72, "bf16", 8)
    v["x"][7, 3] = np.nan
    t = {n: R.dev(v[n], "bf16") for n in ("x", "w", "b")}
    for act in range(5):
        y = torch.empty(40, 72, dtype=torch.bfloat16, device="cuda")
        ws, _ = workspace(40, 64, 72, "bf16")
        moe.moe_linear_fwd(t["x"], t["w"], t["b"], y, act, workspace=ws)
        torch.cuda.synchronize()
        bad = torch.isnan(y).cpu().numpy()
        assert bad[7].all() and not np.delete(bad, 7, axis=0).any()


def test_rows_past_32_bits():
    """More than 2^31 outputs and inputs: the last rows of each."""
    T, I, O = (1 << 31) // 2048 + 300, 2048, 64  # noqa: E741
    for T, I, O in ((T, I, O), (T, O, I)):  # noqa: E741
        note(f"linear T={T} I={I} O={O}")
        v = inputs(300, I, O, "bf16", 12)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        x, dy, z = torch.zeros(T, I, **bf), torch.zeros(T, O, **bf), torch.zeros(T, O, **bf)
        x[-300:], dy[-300:], z[-300:] = R.dev(v["x"], "bf16"), R.dev(v["dy"], "bf16"), R.dev(v["z"], "bf16")
        w, b = R.dev(v["w"], "bf16"), R.dev(v["b"], "bf16")
        y = torch.empty(T, O, **bf)
        ws = torch.empty(max(16, moe.moe_linear_workspace_bytes(T, I, O, torch.bfloat16)), dtype=torch.uint8, device="cuda")
        moe.moe_linear_fwd(x, w, b, y, R.SILU, workspace=ws)
        torch.cuda.synchronize()
        ry, _ = R.linear(v["x"], v["w"], v["b"], R.SILU)
        size = np.abs(v["x"]) @ np.abs(v["w"]) + np.abs(v["b"])
        R.within("y", R.host(y[-300:]), ry, 2.0 ** -8 * np.abs(ry) + 1.2 * (I + 40) * 2.0 ** -23 * size)
        first = R.act(R.SILU, v["b"])  # rows of zeros
        R.within("y of zeros", R.host(y[:5]), np.tile(first, (5, 1)), 2.0 ** -8 * np.abs(first) + 1e-6)
        dx, dw = torch.empty(T, I, **bf), torch.empty_like(w)
        moe.moe_linear_bwd(x, w, dy, y, dx, dw, None, R.SILU, z, workspace=ws)
        torch.cuda.synchronize()
        rz, _ = R.linear_dz(v["z"], None, v["dy"], R.SILU)
        slip = 2.0 ** -8 * np.abs(rz) + 40 * 2.0 ** -24 * np.abs(v["dy"]) * (1 + np.abs(v["z"]))
        ref, size = rz @ v["w"].T, np.abs(rz) @ np.abs(v["w"].T)
        R.within("dx", R.host(dx[-300:]), ref, 2.0 ** -8 * np.abs(ref) + (O + 2) * 2.0 ** -23 * size + 1.01 * slip @ np.abs(v["w"].T))
        ref, size = v["x"].T @ rz, np.abs(v["x"].T) @ np.abs(rz)
        R.within("dw", R.host(dw), ref, 2.0 ** -8 * np.abs(ref) + 302 * 2.0 ** -23 * size + 1.01 * np.abs(v["x"].T) @ slip)
        assert (dx[:-300] == 0).all()


def test_more_rows_than_one_grid_row():
    """2^30 narrow rows: more than 2^32 threads.  Only the last 200 rows are not zero."""
    T, I, O, n = 1 << 30, 8, 8, 200  # noqa: E741
    note(f"linear T={T} I={I} O={O}")
    v = inputs(n, I, O, "bf16", 15)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, dy = torch.zeros(T, I, **bf), torch.zeros(T, O, **bf)
    x[-n:], dy[-n:] = R.dev(v["x"], "bf16"), R.dev(v["dy"], "bf16")
    w, b = R.dev(v["w"], "bf16"), R.dev(v["b"], "bf16")
    ws = torch.empty(max(16, moe.moe_linear_workspace_bytes(T, I, O, torch.bfloat16)), dtype=torch.uint8, device="cuda")
    y = torch.full((T, O), 7.0, **bf)
    moe.moe_linear_fwd(x, w, b, y, workspace=ws)
    torch.cuda.synchronize()
    ref, size = v["x"] @ v["w"] + v["b"], np.abs(v["x"]) @ np.abs(v["w"]) + np.abs(v["b"])
    R.within("y", R.host(y[-n:]), ref, 2.0 ** -8 * np.abs(ref) + (I + 2) * 2.0 ** -23 * size)
    assert (y[:-n] == b).all()  # rows of zeros: the bias, which is in bf16
    dw = torch.empty_like(w)
    moe.moe_linear_bwd(x, w, dy, None, y, dw, workspace=ws)
    torch.cuda.synchronize()
    ref, size = v["dy"] @ v["w"].T, np.abs(v["dy"]) @ np.abs(v["w"].T)
    R.within("dx", R.host(y[-n:]), ref, 2.0 ** -8 * np.abs(ref) + (O + 2) * 2.0 ** -23 * size)
    assert (y[:-n] == 0).all()
    ref, size = v["x"].T @ v["dy"], np.abs(v["x"].T) @ np.abs(v["dy"])
    R.within("dw", R.host(dw), ref, 2.0 ** -8 * np.abs(ref) + (n + 2) * 2.0 ** -23 * size)


def test_rows_behind_the_last_are_left():
    v = inputs(40, 72, 136, "bf16", 13)
    t = {n: R.dev(v[n], "bf16") for n in ("x", "w", "b", "dy")}
    y = torch.full((60, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((60, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    ws, need = workspace(40, 72, 136, "bf16")
    moe.moe_linear_fwd(t["x"], t["w"], t["b"], y[:40], workspace=ws[:need])
    moe.moe_linear_bwd(t["x"], t["w"], t["dy"], None, dx[:40], None, workspace=ws[:need])
    torch.cuda.synchronize()
    assert (y[40:] == 7.0).all() and (dx[40:] == 7.0).all()
