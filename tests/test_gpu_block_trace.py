"""Every kernel of the block operators is a launch of its own in the trace."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import (
    FFNWorkspace, W4Experts, W4Linear, ffn_backward, ffn_forward, layer_norm_backward, layer_norm_forward, quantize_w4)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _names(fn):
    with B.KernelTrace(16) as t:
        out = fn()
    torch.cuda.synchronize()
    assert all(ms >= 0.0 for _, ms in t.durations_ms()) and t.count == len(t.names)
    return t.names, out


def test_one_record_per_kernel():
    build.build()
    for rows, H in ((2000, 768), (50, 333), (3, 70)):  # persistent blocks, a block a row, a warp a row
        x = torch.randn(rows, H, device="cuda")
        w = torch.ones(H, device="cuda")
        names, (y, mean, rstd) = _names(lambda: layer_norm_forward(x, w, w))
        assert names == ["layer_norm_fwd"]
        names, _ = _names(lambda: layer_norm_backward(y, x, w, mean, rstd))
        assert names == ["layer_norm_bwd", "layer_norm_bwd_join"]
    x, w = torch.randn(2, 40000, device="cuda"), torch.ones(40000, device="cuda")  # long rows
    names, (y, mean, rstd) = _names(lambda: layer_norm_forward(x, w, w))
    assert names == ["layer_norm_fwd"]
    names, _ = _names(lambda: layer_norm_backward(y, x, w, mean, rstd))
    assert names == ["layer_norm_bwd", "layer_norm_bwd_cols", "layer_norm_bwd_join"]

    W1, W2 = torch.randn(4, 256, 256, device="cuda").to(BF), torch.randn(4, 128, 256, device="cuda").to(BF)
    names, (q, sf) = _names(lambda: quantize_w4(W1, 64))
    assert names == ["quantize_w4"]
    x = torch.randn(3, 256, device="cuda").to(BF)
    names, _ = _names(lambda: W4Linear(q[0], sf[0], 64)(x))
    assert names == ["matvec_w4"]
    ex = W4Experts.quantize(W1, W2, 64)
    idx, w = torch.tensor([[0, 1], [2, 1], [3, 0]], dtype=torch.int32, device="cuda"), torch.ones(3, 2, device="cuda")
    names, _ = _names(lambda: ex(x, idx, w))
    assert names == ["experts_w4_gate_up", "experts_w4_down", "experts_w4_combine"]
    one = W4Experts.quantize(W1[:1], W2[:1], 64)
    names, _ = _names(lambda: one(x))
    assert names == ["experts_w4_gate_up", "experts_w4_down"]

    ws = FFNWorkspace(300, 256, 128)
    x, dy = torch.randn(2, 300, 256, device="cuda").to(BF)
    names, _ = _names(lambda: ffn_forward(x, W1[0], W2[0], ws))
    assert names == ["ffn_gate_up", "ffn_down"]
    names, _ = _names(lambda: ffn_backward(dy, x, W1[0], W2[0], ws))
    assert names == ["ffn_dgate", "ffn_grads"]
