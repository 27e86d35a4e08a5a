"""Forward-mode differentiation through the block operators on the GPU: refused, with gradients enabled and without."""
import pytest
import torch
from torch.autograd import forward_ad

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import gated_ffn, layer_norm, linear, residual_norm

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


@pytest.mark.parametrize("grad", [False, True])
def test_a_tangent_is_refused(grad):
    x, W, w = torch.randn(4, 64, device="cuda").to(BF), torch.randn(64, 64, device="cuda").to(BF), torch.ones(64, device="cuda")
    W1 = torch.randn(64, 128, device="cuda").to(BF)
    calls = (lambda v: gated_ffn(v, W1, W), lambda v: linear(v, W), lambda v: linear(x, W, residual=v), lambda v: layer_norm(v, w),
             lambda v: residual_norm(v, x, w)[0], lambda v: residual_norm(x, v, w)[1])
    with torch.set_grad_enabled(grad):
        for f in calls:
            want = f(x)
            with forward_ad.dual_level():
                assert torch.equal(f(x), want)
                with pytest.raises(NotImplementedError):
                    f(forward_ad.make_dual(x, torch.ones_like(x)))
