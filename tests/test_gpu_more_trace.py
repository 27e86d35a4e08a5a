"""Every kernel of the linear layer, the joint and the decoding layer is a launch of its own in the trace."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import (
    linear_backward, linear_forward, residual_norm_backward, residual_norm_forward)
from routed_grouped_gemm_routing_gb300.layer import DecodeLayer

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _names(fn):
    with B.KernelTrace(16) as t:
        out = fn()
    torch.cuda.synchronize()
    assert all(ms >= 0.0 for _, ms in t.durations_ms()) and t.count == len(t.names)
    return t.names, out


def _r(*shape):
    return torch.randn(shape, device="cuda").to(BF)


def test_linear():
    build.build()
    W, b = _r(2048, 256), _r(256)
    for T, fwd in ((3, ["linear_few"]), (300, ["linear", "linear_join"]), (40000, ["linear"])):
        x, dy = _r(T, 2048), _r(T, 256)
        names, (y, z) = _names(lambda: linear_forward(x, W, b, dy, "silu", for_backward=True))
        assert names == fwd
        grads = ["linear_dw", "linear_join", "linear_grads"] if T == 40000 else ["linear_grads"]  # dW: deep, few tiles
        names, _ = _names(lambda: linear_backward(dy, x, W, z, b, "silu"))
        assert names == (["linear_dz"] if T == 3 else ["linear_dz", "linear_db"]) + grads
        names, _ = _names(lambda: linear_backward(dy, x, W, None, b))
        assert names == (["linear_grads", "linear_dz", "linear_db"] if T == 300 else (["linear_dz"] if T == 3 else ["linear_dz", "linear_db"]) + grads)
        names, _ = _names(lambda: linear_backward(dy, x, W))
        assert names == grads


def test_joint():
    w = torch.ones(300, device="cuda")
    for H in (300, 299):
        o, r = _r(50, H), _r(50, H)
        names, (s, n, st) = _names(lambda: residual_norm_forward(o, r, w[:H]))
        assert names == ["residual_norm_fwd"]
        names, _ = _names(lambda: residual_norm_backward(s, n, o, r, w[:H], st))
        assert names == ["residual_norm_bwd"]  # few rows: one cluster
        o, r = _r(800, H), _r(800, H)
        s, n, st = residual_norm_forward(o, r, w[:H])
        names, _ = _names(lambda: residual_norm_backward(s, n, o, r, w[:H], st))
        assert names == ["residual_norm_bwd", "residual_norm_join"]
    w = torch.ones(9000, device="cuda")  # long rows
    o, r = _r(5, 9000), _r(5, 9000)
    names, (s, n, st) = _names(lambda: residual_norm_forward(o, r, w))
    assert names == ["residual_norm_fwd"]
    names, _ = _names(lambda: residual_norm_backward(s, n, o, r, w, st))
    assert names == ["residual_norm_bwd", "residual_norm_join"]


def test_decode():
    x, R, W1, W2 = _r(3, 64), _r(64, 8), _r(8, 64, 128), _r(8, 64, 64)
    names, (_, idx, w) = _names(lambda: DecodeLayer(R, W1, W2, 2)(x, return_routing=True))
    assert names == ["decode_router", "decode_experts"]
    names, _ = _names(lambda: DecodeLayer(None, W1, W2, 2)(x, idx, w))
    assert names == ["decode_experts"]
