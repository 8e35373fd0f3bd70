"""moe_router_bwd_dlogits refuses outputs and workspaces on buffers that it still
reads: dW_r and its partial sums are written before dx's product reads dlogits and W_r."""
import ctypes

import pytest
import torch

from test_block_abi_cpu import NULL, P, lib, refuses  # noqa: F401 (a fixture)

# an accepted call would run on dummy addresses
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a GPU")
X, W_R, DL, DW, DX, WS = 4, 5, 6, 7, 8, 10


def inside(i, by):
    return ctypes.c_void_p(P(i).value + by)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T,H,E", [(4096, 64, 8), (16, 64, 256)])
def test_overlaps(lib, dtype, T, H, E):  # noqa: F811
    ws = lib.moe_router_workspace_bytes(T, H, E)
    es = 2 if dtype else 4
    ok = [T, H, E, dtype, P(0), P(1), P(2), P(3), P(4), 1, P(5), max(ws, 16), NULL]
    cases = [({DW: P(0)}, 1, "dw_r overlaps x"), ({DW: P(1)}, 1, "dw_r overlaps w_r"), ({DW: P(2)}, 1, "dw_r overlaps dlogits"),
             ({DW: P(4)}, 1, "dw_r overlaps dx"), ({DX: P(1)}, 1, "dx overlaps w_r"), ({DX: P(2)}, 1, "dx overlaps dlogits"),
             ({DW: inside(0, T * H * es - 16)}, 1, "dw_r overlaps x"), ({DX: inside(2, T * E * 4 - 16)}, 1, "dx overlaps dlogits"),
             ({WS: inside(0, 8)}, 1, "workspace must be 16-byte")]
    if ws:
        cases += [({WS: P(i)}, 1, f"workspace overlaps {n}") for i, n in enumerate(("x", "w_r", "dlogits", "dw_r", "dx"))]
        cases += [({WS: inside(3, H * E * es - 16)}, 1, "workspace overlaps dw_r"), ({11: ws - 1}, 3, "workspace")]
    refuses(lib, lib.moe_router_bwd_dlogits, ok, cases)


def test_both_kinds_of_size_are_there(lib):  # noqa: F811
    assert lib.moe_router_workspace_bytes(4096, 64, 8) > 0 and lib.moe_router_workspace_bytes(16, 64, 256) == 0


@pytest.mark.parametrize("at,to", [(DX, P(0)), (WS, inside(3, 256)), (WS, NULL)])
def test_what_is_allowed_passes_the_checks(lib, at, to):  # noqa: F811
    """dx on x; where no workspace is needed, none or one that lies anywhere: on to the launch, which finds no GPU."""
    args = [16, 64, 256, 1, P(0), P(1), P(2), P(3), P(4), 1, P(5), 16, NULL]
    args[at] = to
    assert lib.moe_router_bwd_dlogits(*args) == 4, lib.moe_last_error()
