"""The rest of a block around the routed experts (``layer.moe_layer``).

``layer_norm`` is the norm in front of the router and the experts.  Each op
has an autograd form and a plain forward / backward pair for callers that run
their own backward pass.  PyTorch only allocates the buffers and supplies the
stream.
"""
from __future__ import annotations

import contextlib

import torch

from . import binding as B


def _on(t):
    """Context in which t's device is current (the library launches there)."""
    if not t.is_cuda:
        raise TypeError("expected CUDA tensors")
    return contextlib.nullcontext() if t.device.index == torch.cuda.current_device() else torch.cuda.device(t.device)


# -------------------------------------------------------------- layer norm
def _norm_dims(x, weight, *others):
    if x.dim() != 2:
        raise ValueError("expected x [rows, H]")
    rows, H = x.shape
    for t in (weight,) + others:
        if t is not None and tuple(t.shape) != (H,):
            raise ValueError(f"expected weight and bias [{H}], got {list(t.shape)}")
    return rows, H


def layer_norm_forward(x, weight, bias=None, eps: float = 1e-5):
    """(y, mean, rstd) of x [rows, H]; mean and rstd (f32 [rows]) are what
    layer_norm_backward reads.  x bf16, f16 or f32, its rows may be strided;
    weight and bias [H] in x's type or f32."""
    rows, H = _norm_dims(x, weight, bias)
    with _on(x):
        y = torch.empty((rows, H), dtype=x.dtype, device=x.device)
        stats = torch.empty((2, rows), dtype=torch.float32, device=x.device)
        mean, rstd = stats[0], stats[1]
        B.moe_layer_norm_forward(x, weight, bias, eps, y, mean, rstd)
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, bias: bool = True):
    """(dx, dweight, dbias) for dy [rows, H]; dbias is None without ``bias``.
    dweight and dbias have weight's type."""
    rows, H = _norm_dims(x, weight)
    with _on(x):
        dx = torch.empty((rows, H), dtype=x.dtype, device=x.device)
        dw = torch.empty((H,), dtype=weight.dtype, device=x.device)
        db = torch.empty_like(dw) if bias else None
        ws = torch.empty((max(B.moe_layer_norm_workspace(rows, H), 4),), dtype=torch.uint8, device=x.device)
        B.moe_layer_norm_backward(dy, x, weight, mean, rstd, dx, dw, db, ws)
    return dx, dw, db


def _rows_of(t, H):
    """t as [rows, H] with contiguous rows, without a copy where its strides allow."""
    t = t.reshape(-1, H)
    ok = (H == 1 or t.stride(1) == 1) and (t.shape[0] <= 1 or t.stride(0) >= H)
    return t if ok else t.contiguous()


class LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        H = x.shape[-1]
        x2 = _rows_of(x, H)
        y, mean, rstd = layer_norm_forward(x2, weight, bias, eps)
        ctx.save_for_backward(x2, weight, mean, rstd)
        ctx.has_bias = bias is not None
        return y.view(x.shape)

    @staticmethod
    def backward(ctx, dy):
        x2, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = layer_norm_backward(_rows_of(dy.to(x2.dtype), x2.shape[1]), x2, weight, mean, rstd, ctx.has_bias)
        return dx.view(dy.shape), dw, db, None


def layer_norm(x, weight, bias=None, eps: float = 1e-5):
    """Layer norm over the last axis of x (any number of leading axes), in
    x's type.  Differentiable in x, weight and bias."""
    return LayerNormFunction.apply(x, weight, bias, float(eps))
