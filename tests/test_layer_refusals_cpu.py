"""What the layer driver refuses before any call of the library: a balance loss whose
gradient no backward would take, moments of sizes that there are not."""
import pytest
import torch

from expert_grouped_gemm_top_amd.layer import AdamWBuffers, BalanceLoss, MoeLayerBuffers

T, H, F, E, K = 8, 16, 8, 4, 2


def layer(balance):
    return MoeLayerBuffers(T, H, F, E, K, torch.float32, "cpu", router=True, balance=balance)


@pytest.mark.parametrize("dbalance", [None, torch.ones(1)])
def test_a_backward_without_the_router_loses_the_balance_loss(dbalance):
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    with pytest.raises(AssertionError, match="balance"):
        layer(BalanceLoss(1.0)).backward(f(T, H), f(E, H, F), f(E, H, F), f(E, F, H), dbalance=dbalance)


def test_a_gradient_of_no_balance_loss():
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    with pytest.raises(AssertionError, match="balance"):
        layer(None).backward(f(T, H), f(E, H, F), f(E, H, F), f(E, F, H), w_r=f(H, E), dbalance=torch.ones(1))


@pytest.mark.parametrize("bits", [16, 4, 0, None])
def test_moments_of_other_sizes(bits):
    """Not taken for 32 bits."""
    p = {"w": torch.zeros(8)}
    with pytest.raises(AssertionError, match="bits"):
        AdamWBuffers(p, p, 1e-3, bits=bits)
