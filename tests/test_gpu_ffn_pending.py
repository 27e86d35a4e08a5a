"""A pending gated_ffn holds what its backward reads, not the scratch."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import gated_ffn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_pending_backwards_hold_saved_state_alone():
    build.build()
    T, H, I, layers = 2048, 64, 2048, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, H), generator=g, device="cuda").to(BF).requires_grad_()
    W1 = (torch.randn((H, 2 * I), generator=g, device="cuda") * H ** -0.5).to(BF).requires_grad_()
    W2 = (torch.randn((I, H), generator=g, device="cuda") * I ** -0.5).to(BF).requires_grad_()
    L = B.moe_ffn_workspace_layout(B.MoeFFNShape(T, H, I, 0.0))
    before = torch.cuda.memory_allocated()
    ys = [gated_ffn(x, W1, W2) for _ in range(layers)]
    held = torch.cuda.memory_allocated() - before
    # the caching allocator rounds each block up to at most 2 MB
    assert held <= layers * (L.saved_bytes + T * H * 2 + 2 * (2 << 20)) < layers * (L.saved_bytes + L.ws_bytes), held
    one = torch.autograd.grad(ys[0].float().sum(), (x, W1, W2), retain_graph=True)
    again = torch.autograd.grad(ys[0].float().sum(), (x, W1, W2))
    rest = torch.autograd.grad(sum(y.float().sum() for y in ys[1:2]), (x, W1, W2))
    for a, b, c in zip(one, again, rest):
        assert torch.equal(a, b) and torch.equal(a, c)
