"""The block operators' gradients are first-order ones: asking for a gradient
of a gradient raises instead of leaving the second-order part out."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import gated_ffn, layer_norm

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def test_second_order_of_the_norm():
    x = torch.randn(6, 40, device="cuda", requires_grad=True)
    w = torch.randn(40, device="cuda", requires_grad=True)
    want = torch.autograd.grad(layer_norm(x, w).square().sum(), x)[0]
    g = torch.autograd.grad(layer_norm(x, w).square().sum(), x, create_graph=True)[0]
    assert torch.equal(g, want)  # the gradient itself is there
    with pytest.raises(RuntimeError):
        (g.square().sum() + x.square().sum()).backward()


def test_second_order_of_the_feed_forward():
    x = torch.randn(6, 64, device="cuda").to(BF).requires_grad_()
    W1 = torch.randn(64, 64, device="cuda").to(BF).requires_grad_()
    W2 = torch.randn(32, 64, device="cuda").to(BF).requires_grad_()
    want = torch.autograd.grad(gated_ffn(x, W1, W2).float().sum(), x)[0]
    g = torch.autograd.grad(gated_ffn(x, W1, W2).float().sum(), x, create_graph=True)[0]
    assert torch.equal(g, want)
    with pytest.raises(RuntimeError):
        (g.float().square().sum() + x.float().square().sum()).backward()
