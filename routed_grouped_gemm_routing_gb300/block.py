"""The rest of a block around the routed experts (``layer.moe_layer``).

``layer_norm`` is the norm in front of the router and the experts.  Each op
has an autograd form and a plain forward / backward pair for callers that run
their own backward pass.  PyTorch only allocates the buffers and supplies the
stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import binding as B


_HERE = contextlib.nullcontext()
_F32, _BF = torch.float32, torch.bfloat16
_TYPES = B._TYPES
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
    if not (torch.is_grad_enabled() and (x.requires_grad or W1.requires_grad or W2.requires_grad)):
        return _ffn_call(x, W1, W2, workspace, clamp, False)[-1].view(x.shape)
    return GatedFFNFunction.apply(x, W1, W2, workspace, clamp)


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
