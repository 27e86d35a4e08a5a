"""Forward-mode differentiation, which the block operators do not have: a tensor with a
tangent is refused, with gradients enabled and without, and never loses it without a
word.  The kernels are stood in for by plain products: nothing here touches a device."""
import pytest
import torch
from torch.autograd import forward_ad

from routed_grouped_gemm_routing_gb300 import block

BF = torch.bfloat16


def _linear_forward(x, W, bias=None, residual=None, activation=None, for_backward=False, workspace=None):
    with torch.no_grad():
        y = x.detach() @ W.detach()
        y = y if bias is None else y + bias.detach()
        return y if residual is None else y + residual.detach(), None


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("which", ["x", "W", "bias", "residual"])
def test_linear_refuses_a_tangent(monkeypatch, grad, which):
    monkeypatch.setattr(block, "linear_forward", _linear_forward)
    t = dict(x=torch.ones(2, 8, dtype=BF), W=torch.ones(8, 16, dtype=BF), bias=torch.ones(16, dtype=BF),
             residual=torch.ones(2, 16, dtype=BF))
    with torch.set_grad_enabled(grad):
        want = block.linear(**t)
        with forward_ad.dual_level():
            assert torch.equal(block.linear(**t), want)  # without a tangent as ever
            dual = {**t, which: forward_ad.make_dual(t[which], torch.ones_like(t[which]))}
            with pytest.raises(NotImplementedError):
                block.linear(**dual)
        assert torch.equal(block.linear(**t), want)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("which", ["x", "W1", "W2"])
def test_gated_ffn_refuses_a_tangent(monkeypatch, grad, which):
    class Workspace:
        def __init__(self, T, H, I, device=None, activation_clamp=0.0, train=True):
            self.shape, self.shape_ref = block.B.MoeFFNShape(T, H, I, activation_clamp), None
            self.train, self.ws, self.generation = train, None, 0

    def forward(x, W1, W2, ws, s, s_ref):
        with torch.no_grad():
            g, u = (x.detach() @ W1.detach()).chunk(2, -1)
            return (torch.nn.functional.silu(g) * u) @ W2.detach()

    monkeypatch.setattr(block, "FFNWorkspace", Workspace)
    monkeypatch.setattr(block, "_ffn_forward", forward)
    t = dict(x=torch.ones(2, 8, dtype=BF), W1=torch.ones(8, 32, dtype=BF), W2=torch.ones(16, 8, dtype=BF))
    with torch.set_grad_enabled(grad):
        want = block.gated_ffn(**t)
        with forward_ad.dual_level():
            assert torch.equal(block.gated_ffn(**t), want)
            with pytest.raises(NotImplementedError):
                block.gated_ffn(**{**t, which: forward_ad.make_dual(t[which], torch.ones_like(t[which]))})
