"""The linear product without a workspace: a forward whose reduction is not split
takes none, and gives what it gives with one."""
import pytest
import torch

import block_ref as R
from expert_grouped_gemm_top_amd import moe
from moe_cases import note
from test_gpu_linear import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,I,O", [(1, 8, 8), (40, 128, 264), (300, 72, 136), (4099, 128, 768)])
def test_forward_without_a_workspace(T, I, O, dtype):  # noqa: E741
    note(f"linear without workspace T={T} I={I} O={O} {dtype}")
    v = {n: R.dev(a, dtype) for n, a in inputs(T, I, O, dtype, T).items()}
    ws = torch.empty(moe.moe_linear_workspace_bytes(T, I, O, R.DT[dtype]), dtype=torch.uint8, device="cuda")
    y = [torch.full((T, O), 7.0, dtype=R.DT[dtype], device="cuda") for _ in range(2)]
    for out, space in zip(y, (ws, None)):
        moe.moe_linear_fwd(v["x"], v["w"], v["b"], out, R.SILU, mul=v["mul"], residual=v["residual"], workspace=space)
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[1]) and not (y[0] == 7.0).all()


def test_split_forward_and_backward_need_one():
    x, w, y = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((8, 8192), (8192, 64), (8, 64)))
    before = moe.moe_launch_count()
    with pytest.raises(moe.MoeError, match="WORKSPACE_TOO_SMALL.*moe_linear_fwd: workspace of 0 bytes"):
        moe.moe_linear_fwd(x, w, None, y)
    with pytest.raises(moe.MoeError, match="WORKSPACE_TOO_SMALL.*moe_linear_bwd: workspace of 0 bytes"):
        moe.moe_linear_bwd(x, w, y, None, torch.empty_like(x), torch.empty_like(w))
    assert moe.moe_launch_count() == before
