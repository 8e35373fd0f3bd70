"""Refusals of the operators around the expert path with real tensors: each call is
valid but for one argument, says which, and launches nothing."""
import pytest
import torch

from expert_grouped_gemm_top_amd import moe

pytestmark = pytest.mark.gpu


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def refused(message, f, *args, **kw):
    before = moe.moe_launch_count()
    with pytest.raises(moe.MoeError, match=message):
        f(*args, **kw)
    assert moe.moe_launch_count() == before


def linear(T=4, I=64, O=64, dtype=torch.float32, **change):  # noqa: E741
    ws = z(max(16, moe.moe_linear_workspace_bytes(T, 64, 64, dtype)), dtype=torch.uint8)
    kw = dict(x=z(T, I, dtype=dtype), w=z(I, O, dtype=dtype), bias=z(O, dtype=dtype), y=z(T, O, dtype=dtype), workspace=ws)
    return {**kw, **change}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear(dtype):
    f, other = moe.moe_linear_fwd, torch.bfloat16 if dtype == torch.float32 else torch.float32
    f(**linear(dtype=dtype))
    refused("O=60 is not a multiple of 8", f, **linear(O=60, dtype=dtype))
    refused("I=60 is not a multiple of 8", f, **linear(I=60, dtype=dtype))
    refused("unknown activation 7", f, **linear(dtype=dtype), act=7)
    refused("unknown activation -1", f, **linear(dtype=dtype), act=-1)
    refused("w has shape|y has shape", f, **linear(dtype=dtype, w=z(32, 64, dtype=dtype)))
    refused("y has shape", f, **linear(dtype=dtype, y=z(4, 32, dtype=dtype)))
    refused("w must be torch", f, **linear(dtype=dtype, w=z(64, 64, dtype=other)))
    refused("x must be contiguous", f, **linear(dtype=dtype, x=z(64, 4, dtype=dtype).t()))
    flat = z(64 * 64 + 8, dtype=dtype)
    refused("w must be 16-byte aligned", f, **linear(dtype=dtype, w=flat[1:1 + 64 * 64].view(64, 64)))
    both = z(4, 64, dtype=dtype)
    refused("y overlaps x", f, **linear(dtype=dtype, x=both, y=both))
    torch.cuda.synchronize()


def test_the_others():
    x, g = z(4, 64), z(64)
    idx, w = z(4, 2, dtype=torch.int32), z(4, 2)
    refused("gamma has shape", moe.moe_layernorm_fwd, x, g[:32], None, z(4, 64))
    refused("x must be contiguous", moe.moe_layernorm_fwd, x[:, :56], g[:56], None, z(4, 56))
    refused("topk_idx must be torch.int32", moe.moe_route_scored, x, None, idx.long(), w, 2)
    refused("topk_idx has shape", moe.moe_route_scored, x, None, idx, w, 3)
    refused("bias has shape", moe.moe_route_scored, x, g[:8], idx, w, 2)
    refused("logits must be torch.float32", moe.moe_route_scored, x.bfloat16(), None, idx, w, 2)
    refused("dg has shape", moe.moe_route_scored_bwd, x, idx, w[:3], z(4, 64))
    w_r, ws = z(64, 8), z(max(16, moe.moe_router_workspace_bytes(4, 64, 8)), dtype=torch.uint8)
    refused("dw_r overlaps w_r", moe.moe_router_bwd_dlogits, x, w_r, z(4, 8), w_r, z(4, 64), True, ws)
