"""The workspace that the linear product asks for (host code): sizes, and the
refusals of calls that would use more than they bring."""
import ctypes

import pytest
import torch

from test_block_abi_cpu import NULL, P, lib, refuses  # noqa: F401 (a fixture)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T,I,O", [(8, 8192, 64), (3, 65536, 64)])
@pytest.mark.skipif(torch.cuda.is_available(), reason="were these sizes not split, the calls would run, on dummy addresses")
def test_a_split_forward_refuses_none(lib, dtype, T, I, O):  # noqa: E741, F811
    ok = [T, I, O, dtype, 4] + [P(i) for i in range(7)] + [NULL, 0, NULL]
    refuses(lib, lib.moe_linear_fwd, ok, [({}, 3, "workspace of 0 bytes"), ({13: 16}, 3, "workspace of 16 bytes")])


def test_an_unsplit_forward_refuses_half_a_workspace(lib):  # noqa: F811
    need = lib.moe_linear_workspace_bytes(300, 72, 136, 1)
    ok = [300, 72, 136, 1, 4] + [P(i) for i in range(8)] + [need, NULL]
    refuses(lib, lib.moe_linear_fwd, ok, [({13: need - 1}, 3, "workspace of"), ({13: 0}, 3, "workspace of"),
                                          ({12: NULL}, 1, "workspace must not be NULL"),
                                          ({12: ctypes.c_void_p(P(7).value + 8)}, 1, "aligned")])


def test_sizes_are_never_zero_and_may_fall_with_more_rows(lib):  # noqa: F811
    size = lambda T: lib.moe_linear_workspace_bytes(T, 4096, 4096, 1)  # noqa: E731
    assert all(size(T) > 0 for T in (1, 8, 64, 512, 4096))
    assert size(64) > size(512)
