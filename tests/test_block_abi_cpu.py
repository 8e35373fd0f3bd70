"""Refusals of the operators around the expert path, on the CPU: the library
validates before any HIP call, and the binding before the library."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "expert_grouped_gemm_top_amd", "libmoe.so")
NULL = None


def P(i):
    """A non-null, aligned dummy, 1 GiB from the next: every call here fails before using it."""
    return ctypes.c_void_p((i + 1) << 30)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    from expert_grouped_gemm_top_amd import moe
    return moe.lib()


def refuses(lib, f, ok, changes):
    """Each change of one or more arguments of the valid call is refused with that status and text."""
    for at, status, text in changes:
        args = list(ok)
        for i, v in at.items():
            args[i] = v
        rc = f(*args)
        assert rc == status and text in lib.moe_last_error().decode(), (at, rc, lib.moe_last_error())


def test_route_scored(lib):
    ok = [64, 128, 8, 0, 8, 4, 2, 1, 1.0, P(0), P(1), P(2), P(3), NULL]
    refuses(lib, lib.moe_route_scored, ok, [
        ({0: 0}, 1, "T=0"), ({2: 129}, 1, "exceeds E"), ({1: 257}, 2, "256"), ({2: 17}, 2, "16"), ({0: 1 << 28}, 2, "2^31"),
        ({3: 2}, 1, "score"), ({4: 0}, 1, "n_groups"), ({4: 3}, 1, "divide"), ({4: 32}, 2, "exceeds 16"), ({5: 0}, 1, "top_groups"),
        ({5: 9}, 1, "top_groups"), ({6: 0}, 1, "group_top"), ({6: 3}, 1, "group_top"),
        ({1: 8, 2: 1, 4: 8, 5: 1, 6: 2}, 1, "group size 1"), ({1: 32, 5: 1, 2: 5}, 1, "4 experts of 1"),
        ({8: float("nan")}, 1, "scale"), ({8: float("inf")}, 1, "scale"),
        ({9: NULL}, 1, "logits"), ({11: NULL}, 1, "topk_idx"), ({12: NULL}, 1, "topk_w"), ({11: P(0)}, 1, "topk_idx overlaps logits"),
        ({12: P(1)}, 1, "topk_w overlaps bias"), ({12: ctypes.c_void_p(P(2).value + 4)}, 1, "topk_idx overlaps topk_w")])


def test_route_scored_bwd(lib):
    ok = [64, 128, 8, 0, 1, 1.0, P(0), P(1), P(2), P(3), NULL]
    refuses(lib, lib.moe_route_scored_bwd, ok, [
        ({0: -1}, 1, "T=-1"), ({2: 0}, 1, "k=0"), ({3: -1}, 1, "score"), ({5: float("inf")}, 1, "scale"), ({6: NULL}, 1, "logits"),
        ({7: NULL}, 1, "topk_idx"), ({8: NULL}, 1, "dg"), ({9: NULL}, 1, "dlogits"), ({9: P(0)}, 1, "dlogits overlaps logits"),
        ({9: ctypes.c_void_p(P(2).value + 64)}, 1, "dlogits overlaps dg")])


def test_router_bwd_dlogits(lib):
    ws = lib.moe_router_workspace_bytes(128, 2048, 128)
    ok = [128, 2048, 128, 1, P(0), P(1), P(2), P(3), P(4), 0, P(5), ws, NULL]
    refuses(lib, lib.moe_router_bwd_dlogits, ok, [
        ({0: 0}, 1, "T=0"), ({1: 100}, 2, "multiple of 8"), ({2: 300}, 2, "256"), ({3: 2}, 1, "dtype"), ({4: NULL}, 1, "x must"),
        ({6: NULL}, 1, "dlogits"), ({7: NULL}, 1, "dw_r"), ({8: NULL}, 1, "dx must"), ({11: ws - 1}, 3, "workspace"),
        ({10: NULL}, 1, "workspace")])


def test_layernorm(lib):
    ok = [64, 2048, 1, 1e-5, P(0), P(1), P(2), P(3), P(4), P(5), NULL]
    refuses(lib, lib.moe_layernorm_fwd, ok, [
        ({0: 0}, 1, "T=0"), ({1: 0}, 1, "H=0"), ({1: 12}, 2, "multiple of 8"), ({1: 16392}, 2, "16384"), ({2: 9}, 1, "dtype"),
        ({3: -1.0}, 1, "eps"), ({3: float("nan")}, 1, "eps"), ({4: NULL}, 1, "x must"), ({5: NULL}, 1, "gamma"), ({7: NULL}, 1, "y must"),
        ({8: NULL}, 1, "mean and rstd"), ({4: ctypes.c_void_p(8)}, 1, "x must be 16-byte"),
        ({6: ctypes.c_void_p(P(2).value + 2)}, 1, "beta must be 16-byte"), ({7: ctypes.c_void_p(P(0).value + 16)}, 1, "y overlaps x"),
        ({7: P(1)}, 1, "y overlaps gamma"), ({8: P(0)}, 1, "mean overlaps x"), ({9: P(4)}, 1, "mean overlaps rstd"),
        ({9: P(2)}, 1, "rstd overlaps beta")])
    ws = lib.moe_layernorm_workspace_bytes(64, 2048)
    assert 0 < ws <= 64 << 20 and lib.moe_layernorm_workspace_bytes(1 << 30, 16384) <= 64 << 20
    assert lib.moe_layernorm_workspace_bytes(0, 64) == 0
    ok = [64, 2048, 1, P(0), P(1), P(2), P(3), P(4), P(5), P(6), P(7), P(8), P(9), ws, NULL]
    refuses(lib, lib.moe_layernorm_bwd, ok, [
        ({0: 0}, 1, "T=0"), ({1: 20}, 2, "multiple of 8"), ({3: NULL}, 1, "x must"), ({5: NULL}, 1, "mean"), ({6: NULL}, 1, "rstd"),
        ({7: NULL}, 1, "dy"), ({9: NULL}, 1, "dx must"), ({10: NULL}, 1, "dgamma"), ({13: ws - 1}, 3, "workspace"), ({12: NULL}, 1, "workspace"),
        ({12: ctypes.c_void_p(24)}, 1, "workspace must be 16-byte"), ({9: P(1)}, 1, "dx overlaps gamma"),
        ({9: ctypes.c_void_p(P(4).value + 32)}, 1, "dx overlaps dy"), ({10: P(0)}, 1, "dgamma overlaps x"),
        ({10: P(8)}, 1, "dgamma overlaps dbeta"), ({11: P(3)}, 1, "dbeta overlaps rstd"), ({12: P(6)}, 1, "workspace overlaps dx"),
        ({12: ctypes.c_void_p(P(2).value + 64)}, 1, "workspace overlaps mean")])


def test_linear_fwd(lib):
    ws = lib.moe_linear_workspace_bytes(64, 256, 128, 1)
    ok = [64, 256, 128, 1, 4] + [P(i) for i in range(8)] + [ws, NULL]
    refuses(lib, lib.moe_linear_fwd, ok, [
        ({0: 0}, 1, "T=0"), ({0: (1 << 30) + 1}, 2, "T=1073741825"), ({0: 1 << 28, 1: 4096}, 2, "too large"), ({1: 20}, 2, "I=20"), ({2: 0}, 1, "O=0"), ({2: 36}, 2, "O=36"), ({1: (1 << 20) + 8}, 2, "exceeds"),
        ({3: 4}, 1, "dtype"), ({4: 5}, 1, "activation"), ({4: -1}, 1, "activation"), ({5: NULL}, 1, "x must"), ({6: NULL}, 1, "w must"),
        ({11: NULL}, 1, "y must"), ({5: ctypes.c_void_p(34)}, 1, "aligned"), ({11: P(0)}, 1, "y overlaps x"),
        ({11: P(1)}, 1, "y overlaps w"), ({11: P(5)}, 1, "y overlaps z_save"), ({10: P(4)}, 1, "z_save overlaps residual"),
        ({11: ctypes.c_void_p(P(4).value + 256)}, 1, "y overlaps residual")])
    if ws:
        refuses(lib, lib.moe_linear_fwd, ok, [({13: ws - 1}, 3, "workspace"), ({12: NULL}, 1, "workspace"),
                                              ({12: P(6)}, 1, "workspace overlaps y")])


def test_linear_bwd(lib):
    ws = lib.moe_linear_workspace_bytes(64, 256, 128, 1)
    assert ws > 0 and lib.moe_linear_workspace_bytes(64, 256, 128, 7) == 0
    # x, w, z, mul, dy, dz, dx_add, dx, dw, dbias, dmul, workspace
    ok = [64, 256, 128, 1, 4] + [P(i) for i in range(12)] + [ws, NULL]
    x, w, z, mul, dy, dz, dx_add, dx, dw, dbias, dmul, wsp = range(5, 17)
    refuses(lib, lib.moe_linear_bwd, ok, [
        ({0: 0}, 1, "T=0"), ({1: 4}, 2, "I=4"), ({4: 9}, 1, "activation"), ({dy: NULL}, 1, "dy must"), ({x: NULL}, 1, "x must"),
        ({w: NULL}, 1, "w must"), ({z: NULL}, 1, "z must"), ({dz: NULL}, 1, "dz must"), ({dmul: NULL}, 1, "mul and dmul"),
        ({mul: NULL}, 1, "mul and dmul"), ({dx: NULL}, 1, "dx_add without"), ({dz: ctypes.c_void_p(P(4).value + 16)}, 1, "dz overlaps dy"),
        ({dx: P(4)}, 1, "dx overlaps dy"), ({dx: P(5)}, 1, "dx overlaps dz"), ({dw: P(1)}, 1, "dw overlaps w"),
        ({dmul: P(5)}, 1, "dmul overlaps dz"), ({dbias: P(2)}, 1, "dbias overlaps z"), ({dx: ctypes.c_void_p(40)}, 1, "aligned"),
        ({17: ws - 1}, 3, "workspace"), ({wsp: NULL}, 1, "workspace"), ({wsp: P(5)}, 1, "workspace overlaps dz"),
        ({dx_add: NULL, dx: NULL, dw: NULL, dbias: NULL, mul: NULL, dmul: NULL}, 1, "no gradient"),
        ({4: 0, z: NULL, dz: NULL, mul: NULL, dmul: NULL, 17: 0}, 3, "workspace")])


def test_the_binding_refuses_before_the_library():
    from expert_grouped_gemm_top_amd import moe
    a = torch.zeros(4, 16)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: moe.moe_route_scored(a, None, i, a[:, :2], 2),
                 lambda: moe.moe_route_scored(None, None, i, a, 2),
                 lambda: moe.moe_route_scored(a[0], None, i, a, 2),
                 lambda: moe.moe_route_scored(a[:0], None, i, a, 2),
                 lambda: moe.moe_route_scored_bwd(a, None, a, a),
                 lambda: moe.moe_router_bwd_dlogits(a, a, a, a, a, True),
                 lambda: moe.moe_layernorm_fwd(a, a[0], None, a),
                 lambda: moe.moe_layernorm_bwd(a, a[0], a[:, 0], a[:, 0], a, a, a[0], None, None),
                 lambda: moe.moe_linear_fwd(a, a.t(), None, a),
                 lambda: moe.moe_linear_fwd(a, None, None, a),
                 lambda: moe.moe_linear_bwd(a, a, a, None, a, a)):
        with pytest.raises(moe.MoeError):
            call()


def test_sizes_that_an_int_cannot_hold():
    from expert_grouped_gemm_top_amd import moe
    for shape in ((2**32 + 8, 8), (8, 2**31)):
        with pytest.raises(moe.MoeError, match="2\\^31"):
            moe._rows(torch.empty(shape, device="meta"), "x")
