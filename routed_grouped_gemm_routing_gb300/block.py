"""The rest of a block around the routed experts (``layer.moe_layer``).

``layer_norm`` is the norm in front of the router and the experts,
``residual_norm`` the joint of two halves of a block, ``linear`` a projection with
what surrounds its product.  Each op has an autograd form and a plain forward /
backward pair for callers that run their own backward pass.  PyTorch only
allocates the buffers and supplies the stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch
from torch.autograd import forward_ad

from . import binding as B


_HERE = contextlib.nullcontext()
_F32, _BF = torch.float32, torch.bfloat16
_TYPES = B._TYPES
_BIAS = (torch.bfloat16, torch.float32)
_current = torch.cuda.current_device
_stream_of = torch._C._cuda_getCurrentRawStream


def _plain(t, dtype, shape, dev):
    """Whether t is a contiguous tensor of that type and shape on device dev."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


# The calls below take a few microseconds on the GPU at decoding sizes, so what
# the host does for one counts.  Each first tries its whole check in one
# expression and calls the library with the pointers; whatever does not pass
# (another device, strided rows, a wrong argument) goes the long way, through
# the binding's checks and their messages.


def _on(t):
    """Context in which t's device is current (the library launches there)."""
    dev = t.get_device()
    if dev < 0:
        raise TypeError("expected CUDA tensors")
    return _HERE if dev == torch.cuda.current_device() else torch.cuda.device(dev)


class _NoSecondOrder(torch.autograd.Function):
    """Passes gradients on; differentiating them raises."""

    @staticmethod
    def forward(ctx, *grads):
        return tuple(g.view_as(g) for g in grads)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the block operators have first-order gradients only")


def _first_order(backward):
    """A backward whose kernels no graph records.  Under create_graph its
    gradients raise when they are differentiated themselves, whatever dy is
    (torch's once_differentiable lets them through where dy is a constant, and
    the second-order part would be missing without a word)."""

    @functools.wraps(backward)
    def wrapped(ctx, dy):
        if not torch.is_grad_enabled():
            return backward(ctx, dy)
        with torch.no_grad():
            out = backward(ctx, dy)
        marked = iter(_NoSecondOrder.apply(*(t.detach().requires_grad_() for t in out if t is not None)))
        return tuple(None if t is None else next(marked) for t in out)

    return wrapped


def _has_tangent(*tensors):
    """Whether one of the tensors carries a tangent of forward-mode differentiation.
    The operators have none: their autograd functions refuse such tensors, which a
    call around those would take without their tangents and without a word."""
    return forward_ad._current_level >= 0 and any(
        t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


# -------------------------------------------------------------- layer norm
def _norm_dims(x, weight, bias=None):
    if x.dim() != 2:
        raise ValueError("expected x [rows, H]")
    rows, H = x.shape
    if weight.shape != (H,) or (bias is not None and bias.shape != (H,)):
        raise ValueError(f"expected weight and bias [{H}]")
    return rows, H


def layer_norm_forward(x, weight, bias=None, eps: float = 1e-5):
    """(y, mean, rstd) of x [rows, H]; mean and rstd (f32 [rows]) are what
    layer_norm_backward reads.  x bf16, f16 or f32, its rows may be strided;
    weight and bias [H] in x's type or f32."""
    dt, wt, sh, d = x.dtype, weight.dtype, x.shape, x.get_device()
    if (len(sh) == 2 and sh[1] <= B.NORM_MAX_H and dt in _TYPES and wt in _TYPES and d >= 0 and d == _current()
            and x.is_contiguous() and _plain(weight, wt, sh[1:], d) and (bias is None or _plain(bias, wt, sh[1:], d))):
        rows, dev = sh[0], x.device
        y = torch.empty_like(x)
        mean = torch.empty((rows,), dtype=_F32, device=dev)
        rstd = torch.empty((rows,), dtype=_F32, device=dev)
        rc = B.lib().moe_layer_norm_forward(
            rows, sh[1], _TYPES[dt], _TYPES[wt], x.data_ptr(), sh[1], weight.data_ptr(),
            None if bias is None else bias.data_ptr(), eps, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _stream_of(d))
        if rc:
            B._check(rc)
        return y, mean, rstd
    rows, H = _norm_dims(x, weight, bias)
    with _on(x):
        dev = x.device
        y = torch.empty((rows, H), dtype=x.dtype, device=dev)
        mean = torch.empty((rows,), dtype=torch.float32, device=dev)
        rstd = torch.empty((rows,), dtype=torch.float32, device=dev)
        B.moe_layer_norm_forward(x, weight, bias, eps, y, mean, rstd)
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, bias: bool = True):
    """(dx, dweight, dbias) for dy [rows, H]; dbias is None without ``bias``.
    dweight and dbias have weight's type."""
    dt, wt, sh, d = x.dtype, weight.dtype, x.shape, x.get_device()
    if (len(sh) == 2 and sh[1] <= B.NORM_MAX_H and dt in _TYPES and wt in _TYPES and d >= 0 and d == _current()
            and x.is_contiguous() and _plain(dy, dt, sh, d) and _plain(weight, wt, sh[1:], d) and _plain(mean, _F32, sh[:1], d)
            and _plain(rstd, _F32, sh[:1], d)):
        rows, H, dev = sh[0], sh[1], x.device
        dx, dw = torch.empty_like(x), torch.empty_like(weight)
        db = torch.empty_like(weight) if bias else None
        ws = torch.empty((B.moe_layer_norm_workspace(rows, H) + 4,), dtype=torch.uint8, device=dev)
        rc = B.lib().moe_layer_norm_backward(
            rows, H, _TYPES[dt], _TYPES[wt], dy.data_ptr(), H, x.data_ptr(), H, weight.data_ptr(), mean.data_ptr(),
            rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(), db.data_ptr() if bias else None, ws.data_ptr(), _stream_of(d))
        if rc:
            B._check(rc)
        return dx, dw, db
    rows, H = _norm_dims(x, weight)
    with _on(x):
        dev = x.device
        dx = torch.empty((rows, H), dtype=x.dtype, device=dev)
        dw = torch.empty((H,), dtype=weight.dtype, device=dev)
        db = torch.empty((H,), dtype=weight.dtype, device=dev) if bias else None
        ws = torch.empty((max(B.moe_layer_norm_workspace(rows, H), 4),), dtype=torch.uint8, device=dev)
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
    @_first_order
    def backward(ctx, dy):
        x2, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = layer_norm_backward(_rows_of(dy.to(x2.dtype), x2.shape[1]), x2, weight, mean, rstd, ctx.has_bias)
        return dx.view(dy.shape), dw, db, None


def layer_norm(x, weight, bias=None, eps: float = 1e-5):
    """Layer norm over the last axis of x (any number of leading axes), in
    x's type.  Differentiable in x, weight and bias, once."""
    return LayerNormFunction.apply(x, weight, bias, float(eps))


# ---------------------------------------------------------- residual joint
def _joint_dims(out, residual, weight, bias, post_weight, post_bias, gate):
    """(rows, H, gate kind) of a call."""
    sh = out.shape
    if len(sh) != 2 or sh != residual.shape:
        raise ValueError(f"expected out and residual [rows, H], got {list(out.shape)} and {list(residual.shape)}")
    rows, H = sh
    hs = sh[1:]
    if (weight.shape != hs or (bias is not None and bias.shape != hs) or (post_weight is not None and post_weight.shape != hs)
            or (post_bias is not None and post_bias.shape != hs)):
        raise ValueError(f"expected weight, bias, post_weight and post_bias [{H}]")
    if post_bias is not None and post_weight is None:
        raise ValueError("post_bias without post_weight")
    if gate is None:
        return rows, H, B.GATE_NONE
    if gate.shape == hs:
        return rows, H, B.GATE_CHANNEL
    if gate.shape != (rows, 1):
        raise ValueError(f"expected gate [{H}] (per channel) or [{rows}, 1] (per token), got {list(gate.shape)}")
    return rows, H, B.GATE_TOKEN


_joint_plans = {}  # of a call's shape and options: shape, reference to it, bytes of the backward's scratch


def _joint_plan(sh, xt, wt, kind, gk, residual_scale, eps):
    key = (sh, xt, wt, kind, gk, residual_scale, eps)
    plan = _joint_plans.get(key)
    if plan is None:
        if len(_joint_plans) >= 1024:  # rows of every length have passed
            _joint_plans.clear()
        s = B.residual_norm_shape(*sh, xt, wt, kind, gk, residual_scale, eps)
        plan = _joint_plans[key] = (s, ctypes.byref(s), B.moe_residual_norm_workspace(s))
    return plan


def _ptr_of(t):
    return None if t is None else t.data_ptr()


def _joint_plain(d, xt, wt, sh, post_weight, post_bias, gate, rows, params):
    """The gate kind of a call whose tensors are all there, contiguous, of the right
    types and shapes and on the current device d; else None, whatever the reason."""
    if d < 0 or d != _current() or len(sh) != 2 or (post_bias is not None and post_weight is None):
        return None
    for t in rows:
        if t is not None and (t.dtype is not xt or t.shape != sh or t.get_device() != d or not t.is_contiguous()):
            return None
    hs = sh[1:]
    for t in params:
        if t is not None and (t.dtype is not wt or t.shape != hs or t.get_device() != d or not t.is_contiguous()):
            return None
    if gate is None:
        return B.GATE_NONE
    if gate.dtype is not wt or gate.get_device() != d or not gate.is_contiguous():
        return None
    return B.GATE_CHANNEL if gate.shape == hs else B.GATE_TOKEN if gate.shape == (sh[0], 1) else None


def residual_norm_forward(out, residual, weight, bias=None, post_weight=None, post_bias=None, gate=None,
                          residual_scale: float = 1.0, eps: float = 1e-5, kind: str = "layer"):
    """(stream, normed, stats) of
        stream = residual_scale residual + gate (norm(out) post_weight + post_bias)
        normed = norm(stream) weight + bias
    for out and residual [rows, H] (bf16, f16 or f32; rows may be strided).
    norm: a layer norm, or with kind "rms" without its means.  Without post_weight
    out goes in as it is.  gate: [H] per channel, [rows, 1] per token, or None.
    Parameters and gate in out's type or all f32.  stats (f32 [4, rows]) is what
    residual_norm_backward reads."""
    xt, wt, d, sh = out.dtype, weight.dtype, out.get_device(), out.shape
    gk = _joint_plain(d, xt, wt, sh, post_weight, post_bias, gate, (out, residual), (weight, bias, post_weight, post_bias))
    if gk is not None:
        rows, H = sh
        ref = _joint_plan(sh, xt, wt, kind, gk, residual_scale, eps)[1]
        stream, normed = torch.empty_like(out), torch.empty_like(out)
        stats = torch.empty((4, rows), dtype=_F32, device=out.device)
        rc = B.lib().moe_residual_norm_forward(
            ref, out.data_ptr(), H, residual.data_ptr(), H, _ptr_of(gate), _ptr_of(post_weight), _ptr_of(post_bias),
            weight.data_ptr(), _ptr_of(bias), stream.data_ptr(), normed.data_ptr(), stats.data_ptr(), _stream_of(d))
        if rc:
            B._check(rc)
        return stream, normed, stats
    rows, H, gk = _joint_dims(out, residual, weight, bias, post_weight, post_bias, gate)
    s = _joint_plan((rows, H), xt, wt, kind, gk, residual_scale, eps)[0]
    with _on(out):
        dev = out.device
        stream = torch.empty((rows, H), dtype=out.dtype, device=dev)
        normed = torch.empty((rows, H), dtype=out.dtype, device=dev)
        stats = torch.empty((4, rows), dtype=_F32, device=dev)
        B.moe_residual_norm_forward(s, out, residual, gate, post_weight, post_bias, weight, bias, stream, normed, stats)
    return stream, normed, stats


def residual_norm_backward(dstream, dnormed, out, residual, weight, stats, bias=None, post_weight=None, post_bias=None,
                           gate=None, residual_scale: float = 1.0, kind: str = "layer"):
    """(dout, dresidual, dweight, dbias, dpost_weight, dpost_bias, dgate) for the
    gradients of both outputs (either may be None), after residual_norm_forward
    on the same arguments; None for a parameter that is not there."""
    xt, wt, d, sh = out.dtype, weight.dtype, out.get_device(), out.shape
    gk = _joint_plain(d, xt, wt, sh, post_weight, post_bias, gate, (out, residual, dstream, dnormed),
                      (weight, bias, post_weight, post_bias))
    if gk is not None and _plain(stats, _F32, (4, sh[0]), d):
        H = sh[1]
        _, ref, size = _joint_plan(sh, xt, wt, kind, gk, residual_scale, 1e-5)
        dout, dres, dw = torch.empty_like(out), torch.empty_like(out), torch.empty_like(weight)
        db, dpw, dpb, dg = (None if p is None else torch.empty_like(p) for p in (bias, post_weight, post_bias, gate))
        ws = torch.empty((size,), dtype=torch.uint8, device=out.device) if size else None
        rc = B.lib().moe_residual_norm_backward(
            ref, _ptr_of(dstream), H, _ptr_of(dnormed), H, out.data_ptr(), H, residual.data_ptr(), H, _ptr_of(gate),
            _ptr_of(post_weight), _ptr_of(post_bias), weight.data_ptr(), stats.data_ptr(), _ptr_of(ws), dout.data_ptr(),
            dres.data_ptr(), dw.data_ptr(), _ptr_of(db), _ptr_of(dpw), _ptr_of(dpb), _ptr_of(dg), _stream_of(d))
        if rc:
            B._check(rc)
        return dout, dres, dw, db, dpw, dpb, dg
    rows, H, gk = _joint_dims(out, residual, weight, bias, post_weight, post_bias, gate)
    for t, n in ((dstream, "dstream"), (dnormed, "dnormed")):
        if t is not None and t.shape != (rows, H):
            raise ValueError(f"expected {n} [{rows}, {H}], got {list(t.shape)}")
    if stats.shape != (4, rows):
        raise ValueError(f"expected the forward's stats [4, {rows}], got {list(stats.shape)}")
    s, _, size = _joint_plan((rows, H), xt, wt, kind, gk, residual_scale, 1e-5)
    with _on(out):
        dev = out.device
        dout = torch.empty((rows, H), dtype=out.dtype, device=dev)
        dres = torch.empty((rows, H), dtype=out.dtype, device=dev)
        dw, db, dpw, dpb, dg = (None if p is None else torch.empty(p.shape, dtype=weight.dtype, device=dev)
                                for p in (weight, bias, post_weight, post_bias, gate))
        ws = torch.empty((size,), dtype=torch.uint8, device=dev) if size else None
        B.moe_residual_norm_backward(s, dstream, dnormed, out, residual, gate, post_weight, post_bias, weight, stats, ws,
                                     dout, dres, dw, db, dpw, dpb, dg)
    return dout, dres, dw, db, dpw, dpb, dg


class ResidualNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, out, residual, weight, bias, post_weight, post_bias, gate, residual_scale, eps, kind):
        ctx.set_materialize_grads(False)
        H = out.shape[-1]
        o2, r2 = _rows_of(out, H), _rows_of(residual, H)
        params = [None if p is None else p.contiguous() for p in (weight, bias, post_weight, post_bias)]
        g2 = gate if gate is None or gate.dim() == 1 else gate.reshape(-1, 1)
        g2 = None if g2 is None else g2.contiguous()
        stream, normed, stats = residual_norm_forward(o2, r2, *params, g2, residual_scale, eps, kind)
        ctx.save_for_backward(o2, r2, *params, g2, stats)
        ctx.options = residual_scale, kind, out.shape, None if gate is None else gate.shape
        return stream.view(out.shape), normed.view(out.shape)

    @staticmethod
    def backward(ctx, dstream, dnormed):
        # the outputs' gradients go through one tuple: _first_order's wrapper takes one
        return ResidualNormFunction._backward(ctx, (dstream, dnormed))

    @staticmethod
    @_first_order
    def _backward(ctx, grads):
        o2, r2, weight, bias, post_weight, post_bias, gate, stats = ctx.saved_tensors
        scale, kind, shape, gate_shape = ctx.options
        ds, dn = (None if t is None else _rows_of(t.to(o2.dtype), o2.shape[1]) for t in grads)
        dout, dres, dw, db, dpw, dpb, dg = residual_norm_backward(
            ds, dn, o2, r2, weight, stats, bias, post_weight, post_bias, gate, scale, kind)
        return (dout.view(shape), dres.view(shape), dw, db, dpw, dpb, None if dg is None else dg.view(gate_shape), None,
                None, None)


def residual_norm(out, residual, weight, bias=None, post_weight=None, post_bias=None, gate=None,
                  residual_scale: float = 1.0, eps: float = 1e-5, kind: str = "layer"):
    """(stream, normed) as residual_norm_forward's, over the last axis of out and
    residual (any number of leading axes; a gate per token has them too, and a
    last axis of 1).  Differentiable in every tensor, once."""
    if out.shape != residual.shape:
        raise ValueError(f"out {list(out.shape)} and residual {list(residual.shape)} differ")
    if gate is not None and gate.dim() != 1 and gate.shape != (*out.shape[:-1], 1):
        raise ValueError(f"expected gate [{out.shape[-1]}] or {[*out.shape[:-1], 1]}, got {list(gate.shape)}")
    return ResidualNormFunction.apply(out, residual, weight, bias, post_weight, post_bias, gate, float(residual_scale),
                                      float(eps), kind)


# ------------------------------------------- dense gated feed-forward block
class FFNWorkspace:
    """Device buffers of one block shape, kept from step to step: what the
    forward saves for its backward (the activation and, with ``train``, h) and
    scratch.  ``generation`` counts the forwards that wrote into it: gated_ffn's
    backward raises if another forward has overwritten the workspace since its
    own, and ffn_backward does where it is given its forward's generation."""

    def __init__(self, T: int, H: int, I: int, device=None, activation_clamp: float = 0.0, train: bool = True):
        self.shape = B.MoeFFNShape(T, H, I, activation_clamp)
        self.shape_ref = ctypes.byref(self.shape)
        self.layout = L = B.moe_ffn_workspace_layout(self.shape)
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.train = train
        self.saved = torch.empty(max(L.saved_bytes if train else L.h, 16), dtype=torch.uint8, device=dev)
        self.device = dev
        self.ws = self._scratch()
        self.ws[:16].zero_()
        self.generation = 0

    def _scratch(self):
        return torch.empty(self.layout.ws_bytes, dtype=torch.uint8, device=self.device)

    def status(self) -> int:
        """The status word (synchronises): nonzero when a kernel gave up on a bounded wait."""
        return int(self.ws[:4].view(torch.int32).item())


def _ffn_check(x, W1, W2, ws):
    s = ws.shape
    T, H, I = s.T, s.H, s.I
    if x.shape != (T, H) or W1.shape != (H, 2 * I) or W2.shape != (I, H):
        raise ValueError(f"expected x [{T}, {H}], W1 [{H}, {2 * I}], W2 [{I}, {H}] for this workspace")


def _ffn_shape(ws, activation_clamp):
    """(shape, reference to it) of ws with another clamp, or its own for None."""
    s = ws.shape
    if activation_clamp is None or activation_clamp == s.activation_clamp:
        return s, ws.shape_ref
    s = B.MoeFFNShape(s.T, s.H, s.I, activation_clamp)
    return s, ctypes.byref(s)


def _ffn_forward(x, W1, W2, ws, s, s_ref):
    d = x.get_device()
    T, H, I = s.T, s.H, s.I
    if (d >= 0 and d == _current() and d == ws.device.index and _plain(x, _BF, (T, H), d)
            and _plain(W1, _BF, (H, 2 * I), d) and _plain(W2, _BF, (I, H), d)):
        y = torch.empty_like(x)
        rc = B.lib().moe_ffn_forward(s_ref, x.data_ptr(), W1.data_ptr(), W2.data_ptr(), int(ws.train),
                                     ws.saved.data_ptr(), ws.ws.data_ptr(), y.data_ptr(), _stream_of(d))
        if rc:
            B._check(rc)
        ws.generation += 1
        return y
    _ffn_check(x, W1, W2, ws)
    with _on(x):
        y = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
        B.moe_ffn_forward(s, x, W1, W2, ws.saved, ws.ws, y, ws.train, layout=ws.layout)
    ws.generation += 1
    return y


def ffn_forward(x, W1, W2, ws: FFNWorkspace):
    """y bf16 [T, H] = (silu(x W1[:, :I]) * (x W1[:, I:])) W2 for contiguous
    bf16 x [T, H], W1 [H, 2I] (gate | up), W2 [I, H]."""
    return _ffn_forward(x, W1, W2, ws, ws.shape, ws.shape_ref)


def _ffn_backward(dy, x, W1, W2, ws, s, generation):
    if generation is not None and ws.generation != generation:
        raise RuntimeError("feed-forward backward: its workspace was overwritten by a later forward (this one wrote "
                           f"generation {generation}, the workspace now holds {ws.generation}); give forwards whose "
                           "backwards are still pending workspaces of their own")
    _ffn_check(x, W1, W2, ws)
    if not ws.train:
        raise ValueError("the workspace was made without train")
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    with _on(x):
        dx, dW1, dW2 = (torch.empty(t.shape, dtype=torch.bfloat16, device=x.device) for t in (x, W1, W2))
        B.moe_ffn_backward(s, dy, x, W1, W2, ws.saved, ws.ws, dx, dW1, dW2, layout=ws.layout)
    return dx, dW1, dW2


def ffn_backward(dy, x, W1, W2, ws: FFNWorkspace, generation: int | None = None):
    """(dx, dW1, dW2) bf16 for dy [T, H], after ffn_forward on the same inputs
    and workspace.  generation: ``ws.generation`` as that forward left it;
    raises if another forward has overwritten the workspace since.  None: the
    caller sees to it that the last forward was this one."""
    return _ffn_backward(dy, x, W1, W2, ws, ws.shape, generation)


def _ffn_call(x, W1, W2, ws, activation_clamp, train):
    """(x [T, H], W1, W2, workspace, shape, y [T, H]) of a gated_ffn call; the
    workspace is ws where its shape and form allow, else a new one."""
    H, I = x.shape[-1], W2.shape[0]
    x, W1, W2 = x.reshape(-1, H).contiguous(), W1.contiguous(), W2.contiguous()
    s = (x.shape[0], H, I)
    if ws is None or (ws.shape.T, ws.shape.H, ws.shape.I) != s or (train and not ws.train):
        clamp = ws.shape.activation_clamp if ws is not None and activation_clamp is None else activation_clamp or 0.0
        ws = FFNWorkspace(*s, device=x.device, activation_clamp=clamp, train=train)
    shape, ref = _ffn_shape(ws, activation_clamp)
    return x, W1, W2, ws, shape, _ffn_forward(x, W1, W2, ws, shape, ref)


class GatedFFNFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W1, W2, ws, activation_clamp):
        given = ws
        x2, W1, W2, ws, shape, y = _ffn_call(x, W1, W2, given, activation_clamp, True)
        if ws is not given:
            ws.ws = None  # what is pending holds the saved values alone; the backward takes scratch of its own
        ctx.save_for_backward(x2, W1, W2)
        ctx.ws, ctx.ws_generation, ctx.clamp = ws, ws.generation, shape.activation_clamp
        return y.view(x.shape)

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        x2, W1, W2 = ctx.saved_tensors
        ws = ctx.ws
        dy2 = dy.to(torch.bfloat16).reshape(x2.shape).contiguous()
        own = ws.ws is None
        if own:
            ws.ws = ws._scratch()  # its status word is not cleared: nobody can read it
        dx, dW1, dW2 = _ffn_backward(dy2, x2, W1, W2, ws, _ffn_shape(ws, ctx.clamp)[0], ctx.ws_generation)
        if own:
            ws.ws = None
        return dx.view(dy.shape), dW1, dW2, None, None


def gated_ffn(x, W1, W2, workspace: FFNWorkspace | None = None, activation_clamp: float | None = None):
    """The dense gated feed-forward block (a shared expert): bf16 x [..., H],
    W1 [H, 2I] (gate | up), W2 [I, H]; H and I multiples of 8.  Differentiable
    in all three, once.  activation_clamp as in ``layer.moe_layer``, for this call
    alone; None: the workspace's, or none without one.  A workspace of another
    shape, or one made without ``train`` where gradients are wanted, is left
    alone and a new one made.  Without gradients (no_grad, or no input that
    requires one) the workspace's form is taken, without one the inference
    form."""
    clamp = None if activation_clamp is None else float(activation_clamp)
    wanted = torch.is_grad_enabled() and (x.requires_grad or W1.requires_grad or W2.requires_grad)
    if not wanted and not _has_tangent(x, W1, W2):
        return _ffn_call(x, W1, W2, workspace, clamp, False)[-1].view(x.shape)
    return GatedFFNFunction.apply(x, W1, W2, workspace, clamp)


# ------------------------------------------------------------ linear layer
@functools.lru_cache(maxsize=256)
def _linear_plan(T, K, N, activation):
    """(shape, reference to it, bytes of the forward's and of the backward's scratch)."""
    s = B.linear_shape(T, K, N, activation)
    return s, ctypes.byref(s), B.moe_linear_workspace(s, False), B.moe_linear_workspace(s, True)


_no_sums = {}  # of a device: scratch of forwards that keep nothing but a status word there


class LinearWorkspace:
    """Scratch of one linear layer's calls, kept from step to step; calls that
    share one must not overlap.  Without one, each call takes scratch of its own
    whose status nobody can read; what a kernel that gave up was to compute is NaN
    either way."""

    def __init__(self, T: int, K: int, N: int, activation=None, device=None):
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.shape = (T, K, N, activation)
        self.ws = torch.empty(max(_linear_plan(*self.shape)[2:]), dtype=torch.uint8, device=dev)
        self.ws[:16].zero_()

    def status(self) -> int:
        """The status word (synchronises): nonzero when a kernel gave up on a bounded wait."""
        return int(self.ws[:4].view(torch.int32).item())


def _linear_ws(workspace, plan_of, size, dev):
    if workspace is None:
        if size > 256:
            return torch.empty((size,), dtype=torch.uint8, device=dev)
        if dev not in _no_sums:
            # (made under a capture it would belong to that graph's memory)
            ws = torch.empty((256,), dtype=torch.uint8, device=dev)
            if torch.cuda.is_current_stream_capturing():
                return ws
            _no_sums[dev] = ws
        return _no_sums[dev]
    if workspace.shape != plan_of:
        raise ValueError(f"the workspace was made for (T, K, N, activation) = {workspace.shape}, the call has {plan_of}")
    return workspace.ws


def _tma_rows(t):
    """t [rows, n] as it is where the kernels' copies can take its rows, else a contiguous copy."""
    ok = (t.stride(1) == 1 and t.data_ptr() % 16 == 0
          and (t.shape[0] <= 1 or (t.stride(0) % 8 == 0 and t.stride(0) >= t.shape[1])))
    if ok:
        return t
    return _whole(t)


def _whole(t):
    """t contiguous from a 16-byte boundary on, without a copy where it is (None stays None)."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _linear_dims(x, W, bias, residual, activation):
    if x.dim() != 2 or W.dim() != 2 or x.shape[1] != W.shape[0]:
        raise ValueError(f"expected x [T, K] and W [K, N], got {list(x.shape)} and {list(W.shape)}")
    T, K, N = x.shape[0], x.shape[1], W.shape[1]
    if bias is not None and bias.shape != (N,):
        raise ValueError(f"expected bias [{N}], got {list(bias.shape)}")
    if residual is not None and residual.shape != (T, N):
        raise ValueError(f"expected residual [{T}, {N}], got {list(residual.shape)}")
    return (T, K, N, activation), _linear_plan(T, K, N, activation)


def linear_forward(x, W, bias=None, residual=None, activation=None, for_backward: bool = False,
                   workspace: LinearWorkspace | None = None):
    """(y, z) of y bf16 [T, N] = act(x W + bias) + residual for bf16 x [T, K], W
    [K, N] (K and N multiples of 8), bias [N] bf16 or f32, residual bf16 [T, N];
    rows of x and residual may be strided by multiples of 8.  activation: None,
    "silu", "gelu" (with erf) or "gelu_tanh".  z = x W + bias f32 [T, N] with
    for_backward and an activation, else None."""
    d, dev, sh, wh = x.get_device(), x.device, x.shape, W.shape
    if (d >= 0 and d == _current() and len(sh) == 2 and len(wh) == 2 and sh[1] == wh[0] and x.dtype is _BF and W.dtype is _BF
            and W.get_device() == d and x.is_contiguous() and W.is_contiguous()
            and (bias is None or (bias.dtype in _BIAS and _plain(bias, bias.dtype, wh[1:], d)))
            and (residual is None or _plain(residual, _BF, (sh[0], wh[1]), d))
            and (workspace is None or workspace.ws.get_device() == d)):
        T, K = sh
        N = wh[1]
        plan_of = T, K, N, activation
        _, ref, size, _ = _linear_plan(*plan_of)
        y = torch.empty((T, N), dtype=_BF, device=dev)
        z = torch.empty((T, N), dtype=_F32, device=dev) if for_backward and activation is not None else None
        rc = B.lib().moe_linear_forward(
            ref, x.data_ptr(), K, W.data_ptr(), _ptr_of(bias), 0 if bias is None else _TYPES[bias.dtype], _ptr_of(residual),
            N, _ptr_of(z), _linear_ws(workspace, plan_of, size, dev).data_ptr(), y.data_ptr(), _stream_of(d))
        if rc:
            B._check(rc)
        return y, z
    plan_of, (s, _, size, _) = _linear_dims(x, W, bias, residual, activation)
    T, K, N, _ = plan_of
    with _on(x):
        y = torch.empty((T, N), dtype=_BF, device=dev)
        z = torch.empty((T, N), dtype=_F32, device=dev) if for_backward and activation is not None else None
        B.moe_linear_forward(s, x, W, bias, residual, z, _linear_ws(workspace, plan_of, size, dev), y)
    return y, z


def linear_backward(dy, x, W, z=None, bias=None, activation=None, want=(True, True),
                    workspace: LinearWorkspace | None = None):
    """(dx, dW, dbias) for dy bf16 [T, N], after linear_forward on the same inputs
    (z: its second output, with for_backward; None without an activation).  dbias
    has bias's type, None without one.  want: whether dx and dW are; None is
    returned for one that is not.  The residual's gradient is dy."""
    d, sh, wh = x.get_device(), x.shape, W.shape
    want_x, want_w = want
    if (d >= 0 and d == _current() and len(sh) == 2 and len(wh) == 2 and sh[1] == wh[0] and x.dtype is _BF and W.dtype is _BF
            and W.get_device() == d and x.is_contiguous() and W.is_contiguous() and _plain(dy, _BF, (sh[0], wh[1]), d)
            and (activation is None or (z is not None and _plain(z, _F32, (sh[0], wh[1]), d)))
            and (bias is None or (bias.dtype in _BIAS and _plain(bias, bias.dtype, wh[1:], d)))
            and (workspace is None or workspace.ws.get_device() == d)):
        T, K = sh
        N = wh[1]
        plan_of = T, K, N, activation
        _, ref, _, size = _linear_plan(*plan_of)
        dx = torch.empty_like(x) if want_x else None
        dW = torch.empty_like(W) if want_w else None
        db = None if bias is None else torch.empty_like(bias)
        rc = B.lib().moe_linear_backward(
            ref, dy.data_ptr(), N, x.data_ptr(), K, W.data_ptr(), None if activation is None else z.data_ptr(),
            _linear_ws(workspace, plan_of, size, x.device).data_ptr(), _ptr_of(dx), _ptr_of(dW), _ptr_of(db),
            0 if db is None else _TYPES[db.dtype], _stream_of(d))
        if rc:
            B._check(rc)
        return dx, dW, db
    plan_of, (s, _, _, size) = _linear_dims(x, W, bias, None, activation)
    T, K, N, _ = plan_of
    if dy.shape != (T, N):
        raise ValueError(f"expected dy [{T}, {N}], got {list(dy.shape)}")
    if activation is not None and (z is None or z.shape != (T, N)):
        raise ValueError("the backward of an activation needs the forward's z (for_backward=True)")
    with _on(x):
        dx = torch.empty((T, K), dtype=_BF, device=x.device) if want_x else None
        dW = torch.empty((K, N), dtype=_BF, device=x.device) if want_w else None
        db = None if bias is None else torch.empty((N,), dtype=bias.dtype, device=x.device)
        ws = _linear_ws(workspace, plan_of, size, x.device)
        B.moe_linear_backward(s, dy, x, W, None if activation is None else z, ws, dx, dW, db)
    return dx, dW, db


class LinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, bias, residual, activation, workspace):
        K, N = x.shape[-1], W.shape[-1]
        x2, W, bias = _tma_rows(x.reshape(-1, K)), _whole(W), _whole(bias)
        r2 = None if residual is None else _tma_rows(residual.reshape(-1, N))
        train = any(ctx.needs_input_grad[:3])
        y, z = linear_forward(x2, W, bias, r2, activation, train, workspace)
        ctx.save_for_backward(x2, W, z, bias)
        ctx.activation, ctx.workspace, ctx.x_shape = activation, workspace, x.shape
        return y.view(*x.shape[:-1], N)

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        x2, W, z, bias = ctx.saved_tensors
        nx, nW, nb, nr = ctx.needs_input_grad[:4]
        dx = dW = db = None
        if nx or nW or nb:
            dy2 = _tma_rows(dy.to(torch.bfloat16).reshape(x2.shape[0], W.shape[1]))
            dx, dW, db = linear_backward(dy2, x2, W, z, bias if nb else None, ctx.activation, (nx, nW), ctx.workspace)
        return None if dx is None else dx.view(ctx.x_shape), dW, db, dy if nr else None, None, None


def linear(x, W, bias=None, residual=None, activation=None, workspace: LinearWorkspace | None = None):
    """act(x W + bias) + residual for bf16 x [..., K], W [K, N] (the layout of the
    layer's weights; K and N multiples of 8), bias [N] bf16 or f32, residual bf16
    [..., N]; activation as in linear_forward.  Differentiable in all four, once."""
    if residual is not None and residual.shape != (*x.shape[:-1], W.shape[-1]):
        raise ValueError(f"expected residual {[*x.shape[:-1], W.shape[-1]]}, got {list(residual.shape)}")
    if not torch.is_grad_enabled() and not _has_tangent(x, W, bias, residual):
        return _no_grad_linear(x, W, bias, residual, activation, workspace)
    return LinearFunction.apply(x, W, bias, residual, activation, workspace)


def _no_grad_linear(x, W, bias, residual, activation, workspace):
    K, N = x.shape[-1], W.shape[-1]
    y, _ = linear_forward(_tma_rows(x.reshape(-1, K)), _whole(W), _whole(bias),
                          None if residual is None else _tma_rows(residual.reshape(-1, N)), activation, False, workspace)
    return y.view(*x.shape[:-1], N)


# ---------------------------------------------------------- 4-bit weights
def quantize_w4(W, group: int = 128):
    """(codes, scales) of W bf16 [K, N] or [E, K, N] (the layout of the layer's
    W1 and W2): codes uint8 [.., N, K // 2], scales bf16 [.., N, K // group]."""
    W3 = W if W.dim() == 3 else W.unsqueeze(0)
    if W3.dim() != 3:
        raise ValueError("expected W [K, N] or [E, K, N]")
    E, K, N = W3.shape
    if group not in (32, 64, 128) or K % 128:
        raise ValueError("group must be 32, 64 or 128, and K a multiple of 128")
    B._w4_sizes(N, K)
    with _on(W):
        q = torch.empty((E, N, K // 2), dtype=torch.uint8, device=W.device)
        sf = torch.empty((E, N, K // group), dtype=torch.bfloat16, device=W.device)
        B.moe_quantize_w4(W3.contiguous(), q, sf, group)
    return (q, sf) if W.dim() == 3 else (q[0], sf[0])


def _check_w4(q, sf, group, *shape):
    K = shape[-1]
    B._w4_sizes(*shape[-2:])
    if tuple(q.shape) != (*shape[:-1], K // 2) or tuple(sf.shape) != (*shape[:-1], K // group):
        raise ValueError(f"expected codes {[*shape[:-1], K // 2]} and scales {[*shape[:-1], K // group]}, "
                         f"got {list(q.shape)} and {list(sf.shape)}")
    if q.dtype != torch.uint8 or sf.dtype != torch.bfloat16 or not q.is_cuda or not sf.is_cuda:
        raise TypeError("codes must be uint8 and scales bfloat16 CUDA tensors")
    if q.get_device() != sf.get_device():
        raise ValueError(f"codes on cuda:{q.get_device()} and scales on cuda:{sf.get_device()}")
    return q.contiguous(), sf.contiguous()


class W4Linear:
    """y = x W^T for W [N, K] held as 4-bit codes with one scale per ``group``
    values of K (quantize_w4), for a few rows of x at a time.  Not
    differentiable."""

    def __init__(self, q, sf, group: int = 128):
        if group not in (32, 64, 128):
            raise ValueError("group must be 32, 64 or 128")
        N, half = q.shape
        self.N, self.K, self.group = N, 2 * half, group
        self.q, self.sf = _check_w4(q, sf, group, N, 2 * half)

    def forward(self, x, out=None):
        """y bf16 [M, N] for x bf16 [M, K]."""
        M, K = x.shape
        d = x.get_device()
        if d >= 0 and d == _current() and d == self.q.get_device() and out is None and _plain(x, _BF, (M, self.K), d):
            y = torch.empty((M, self.N), dtype=_BF, device=x.device)
            rc = B.lib().moe_matvec_w4(M, self.N, K, self.group, x.data_ptr(), self.q.data_ptr(), self.sf.data_ptr(),
                                       y.data_ptr(), _stream_of(d))
            if rc:
                B._check(rc)
            return y
        if K != self.K:
            raise ValueError(f"x has {K} columns, the weight {self.K}")
        with _on(x):
            if out is None:
                out = torch.empty((M, self.N), dtype=torch.bfloat16, device=x.device)
            B.moe_matvec_w4(x if x.is_contiguous() else x.contiguous(), self.q, self.sf, out, self.group)
        return out

    __call__ = forward


class W4Experts:
    """The layer's experts with 4-bit weights, for decoding: W1 codes
    [E, 2I, H // 2] (gate rows, then up rows), W2 codes [E, H, I // 2], scales
    per ``group``.  E = 1 without routing is a shared expert.
    activation_clamp as in ``layer.moe_layer``.  Not differentiable."""

    def __init__(self, W1_q, W1_sf, W2_q, W2_sf, group: int = 128, activation_clamp: float = 0.0):
        if group not in (32, 64, 128):
            raise ValueError("group must be 32, 64 or 128")
        E, I2, half = W1_q.shape
        self.E, self.H, self.I, self.group = E, 2 * half, I2 // 2, group
        self.W1_q, self.W1_sf = _check_w4(W1_q, W1_sf, group, E, I2, self.H)
        self.W2_q, self.W2_sf = _check_w4(W2_q, W2_sf, group, E, self.H, self.I)
        if self.W1_q.get_device() != self.W2_q.get_device():
            raise ValueError(f"W1 on cuda:{self.W1_q.get_device()} and W2 on cuda:{self.W2_q.get_device()}")
        self.activation_clamp = float(activation_clamp)
        self._sizes = {}  # (T, k) -> shape, workspace bytes

    def _size(self, T, k):
        if (T, k) not in self._sizes:
            s = B.MoeW4Shape(T, self.H, self.I, self.E, k, self.group, self.activation_clamp)
            self._sizes[T, k] = (s, ctypes.byref(s), max(B.moe_w4_workspace(s), 16))
        return self._sizes[T, k]

    @classmethod
    def quantize(cls, W1, W2, group: int = 128, activation_clamp: float = 0.0):
        """From bf16 W1 [E, H, 2I] (gate | up) and W2 [E, I, H]; a shared
        expert's may lack the leading axis."""
        W1, W2 = (W if W.dim() == 3 else W.unsqueeze(0) for W in (W1, W2))
        return cls(*quantize_w4(W1, group), *quantize_w4(W2, group), group, activation_clamp)

    def forward(self, x, topk_idx=None, topk_w=None, out=None):
        """y bf16 [T, H] for x bf16 [T, H] and the routing (topk_idx int
        [T, k], topk_w float [T, k]; neither with a single expert)."""
        T, H = x.shape
        d = x.get_device()
        if (d >= 0 and d == _current() and d == self.W1_q.get_device() and out is None and topk_idx is not None
                and topk_w is not None and _plain(x, _BF, (T, self.H), d)
                and _plain(topk_idx, torch.int32, topk_w.shape, d) and _plain(topk_w, _F32, (T, topk_w.shape[-1]), d)):
            _, ref, size = self._size(T, topk_w.shape[-1])
            dev = x.device
            ws = torch.empty((size,), dtype=torch.uint8, device=dev)
            y = torch.empty_like(x)
            rc = B.lib().moe_forward_w4(
                ref, x.data_ptr(), self.W1_q.data_ptr(), self.W1_sf.data_ptr(), self.W2_q.data_ptr(),
                self.W2_sf.data_ptr(), topk_idx.data_ptr(), topk_w.data_ptr(), ws.data_ptr(), y.data_ptr(), _stream_of(d))
            if rc:
                B._check(rc)
            return y
        if H != self.H:
            raise ValueError("x's hidden size differs from the weights'")
        if topk_idx is None:
            if self.E != 1:
                raise ValueError("several experts need topk_idx and topk_w")
            k = 1
        else:
            k = topk_idx.shape[1]
            if topk_idx.shape != (T, k) or topk_w is None or topk_w.shape != (T, k):
                raise ValueError("expected topk_idx and topk_w [T, k]")
            if topk_idx.dtype is not torch.int32 or not topk_idx.is_contiguous():
                topk_idx = topk_idx.to(torch.int32).contiguous()
            if topk_w.dtype is not torch.float32 or not topk_w.is_contiguous():
                topk_w = topk_w.to(torch.float32).contiguous()
        s, _, size = self._size(T, k)
        with _on(x):
            ws = torch.empty((size,), dtype=torch.uint8, device=x.device)
            if out is None:
                out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
            B.moe_forward_w4(s, x if x.is_contiguous() else x.contiguous(), self.W1_q, self.W1_sf, self.W2_q,
                             self.W2_sf, topk_idx, topk_w, ws, out)
        return out

    __call__ = forward
