"""User-facing routed MoE expert layer.

``moe_layer(x, W1, W2, topk_idx, topk_weights)`` is the single autograd op of
the pages' design (Primus-Turbo "Mega MoE" README, "Key points": one op that
takes external routing).  Forward calls the routing prologue and the
forward entry point of the C ABI; backward calls the backward entry point.
PyTorch only allocates the buffers and supplies the stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import binding as B


class MoEWorkspace:
    """Caller-owned device buffers of one layer shape (reused across steps).

    The routing tables and the saved activations of a forward live in the
    workspace until its backward reads them.  ``generation`` counts the
    forwards that wrote into it: a backward raises if another forward has
    overwritten the workspace since its own forward (two micro-batches or two
    layers sharing one workspace before their backwards)."""

    def __init__(self, T: int, H: int, I: int, E: int, k: int, device=None, activation_clamp: float = 0.0):
        self.shape = B.shape_of(T, H, I, E, k, activation_clamp=activation_clamp)
        self.layout = B.moe_workspace_layout(self.shape)
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        L = self.layout
        self.route = torch.empty(max(L.route_bytes, 16), dtype=torch.uint8, device=dev)
        self.saved = torch.empty(max(L.saved_bytes, 16), dtype=torch.uint8, device=dev)
        self._bwd = None
        self.device = dev
        self.generation = 0

    @property
    def bwd(self):
        if self._bwd is None:
            self._bwd = torch.empty(max(self.layout.bwd_bytes, 16), dtype=torch.uint8, device=self.device)
        return self._bwd


def _dims(x, W1, W2, topk_idx):
    T, H = x.shape
    E, H1, I2 = W1.shape
    if H1 != H or I2 % 2 or tuple(W2.shape) != (E, I2 // 2, H):
        raise ValueError("expected x [T,H], W1 [E,H,2I], W2 [E,I,H]")
    return T, H, I2 // 2, E, topk_idx.shape[1]


class MoEFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W1, W2, topk_idx, topk_weights, ws=None, activation_clamp=0.0, main_grad=False):
        T, H, I, E, k = _dims(x, W1, W2, topk_idx)
        if ws is None or (ws.shape.T, ws.shape.H, ws.shape.I, ws.shape.E, ws.shape.k) != (T, H, I, E, k):
            ws = MoEWorkspace(T, H, I, E, k, device=x.device, activation_clamp=activation_clamp)
        elif ws.shape.activation_clamp != activation_clamp:
            ws.shape.activation_clamp = activation_clamp
        idx = topk_idx if topk_idx.dtype == torch.int32 else topk_idx.to(torch.int32)
        idx = idx.contiguous()
        w = topk_weights.to(torch.float32).contiguous()
        x = x.contiguous()
        y = torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
        B.moe_route_prologue(ws.shape, idx, ws.route)
        B.moe_forward(ws.shape, x, W1.contiguous(), W2.contiguous(), w, ws.route, ws.saved, y)
        ws.generation += 1
        ctx.save_for_backward(x, W1, W2, w)
        ctx.ws = ws
        ctx.ws_generation = ws.generation
        ctx.w_dtype = topk_weights.dtype
        ctx.main_grad = main_grad
        return y

    @staticmethod
    def backward(ctx, dy):
        x, W1, W2, w = ctx.saved_tensors
        ws = ctx.ws
        if ws.generation != ctx.ws_generation:
            raise RuntimeError(
                "moe_layer backward: its workspace was overwritten by a later forward (this forward wrote "
                f"generation {ctx.ws_generation}, the workspace now holds generation {ws.generation}); give "
                "forwards whose backwards are still pending workspaces of their own")
        s = ws.shape
        dev = x.device
        dx = torch.empty_like(x)
        dw = torch.empty(s.T, s.k, dtype=torch.float32, device=dev)
        if ctx.main_grad:
            # FP32 main gradients: W.main_grad += dW; no bf16 gradient
            B.moe_backward_main_grad(s, dy.to(torch.bfloat16).contiguous(), x, W1.contiguous(), W2.contiguous(), w,
                                     ws.route, ws.saved, ws.bwd, dx, W1.main_grad, W2.main_grad, dw)
            return dx, None, None, None, dw.to(ctx.w_dtype), None, None, None
        dW1 = torch.empty_like(W1)
        dW2 = torch.empty_like(W2)
        B.moe_backward(s, dy.to(torch.bfloat16).contiguous(), x, W1.contiguous(), W2.contiguous(), w, ws.route,
                       ws.saved, ws.bwd, dx, dW1, dW2, dw)
        return dx, dW1, dW2, None, dw.to(ctx.w_dtype), None, None, None


def moe_layer(x, W1, W2, topk_idx, topk_weights, workspace: MoEWorkspace | None = None,
              activation_clamp: float = 0.0, accumulate_main_grad: bool = False):
    """y = sum_j topk_weights[:, j] * SwiGLU-MLP_{topk_idx[:, j]}(x), bf16.

    x bf16 [T,H]; W1 bf16 [E,H,2I] (gate | up); W2 bf16 [E,I,H];
    topk_idx int32/int64 [T,k] (-1 = dropped slot); topk_weights float [T,k].
    Differentiable in x, W1, W2 and topk_weights.  activation_clamp > 0
    clamps both SwiGLU inputs to [-c, c] (gradients pass inside only).
    accumulate_main_grad: W1.main_grad and W2.main_grad (float32 tensors of
    W1's and W2's shapes, set by the caller) get += dW1 / dW2 in FP32 and the
    autograd gradients of W1 and W2 are None."""
    if accumulate_main_grad:
        for n, W in (("W1", W1), ("W2", W2)):
            mg = getattr(W, "main_grad", None)
            if mg is None or mg.dtype != torch.float32 or tuple(mg.shape) != tuple(W.shape):
                raise ValueError(f"accumulate_main_grad needs {n}.main_grad: float32 of {n}'s shape")
    with torch.cuda.device(x.device):
        return MoEFunction.apply(x, W1, W2, topk_idx, topk_weights, workspace, float(activation_clamp),
                                 bool(accumulate_main_grad))


class FP8Experts:
    """The layer's expert weights in FP8 for inference (DeepGEMM Mega-MoE
    article, "Code Example: Fused Overlap Path": the weights are transformed
    once, the activations cast per token before each call).

    Built once from bf16 W1 [E,H,2I] and W2 [E,I,H] (moe_quantize_weights_fp8,
    moe_quantize_w2_fp8); ``forward`` casts x (moe_quantize_fp8), builds the
    routing tables and runs moe_forward_fp8.  Needs H and I multiples of 128.
    Not differentiable."""

    def __init__(self, W1, W2):
        E, H, I2 = W1.shape
        I = I2 // 2
        if I2 % 2 or tuple(W2.shape) != (E, I, H):
            raise ValueError("expected W1 [E,H,2I], W2 [E,I,H]")
        if H % 128 or I % 128:
            raise ValueError("the FP8 path needs H and I to be multiples of 128")
        self.E, self.H, self.I = E, H, I
        dev = W1.device
        s = B.shape_of(1, H, I, E, 1)
        self.W1_fp8 = torch.empty(E, 2 * I, H, dtype=torch.uint8, device=dev)
        self.W1_sf = torch.empty(E * 2 * I * H // 32, dtype=torch.uint8, device=dev)
        self.W2_fp8 = torch.empty(E, H, I, dtype=torch.uint8, device=dev)
        self.W2_sf = torch.empty(E * H * I // 32, dtype=torch.uint8, device=dev)
        with torch.cuda.device(dev):
            B.moe_quantize_weights_fp8(s, W1.contiguous(), self.W1_fp8, self.W1_sf)
            B.moe_quantize_w2_fp8(s, W2.contiguous(), self.W2_fp8, self.W2_sf)

    def forward(self, x, topk_idx, topk_weights, workspace: MoEWorkspace | None = None):
        """y bf16 [T,H] of the FP8 layer for x bf16 [T,H] and the routing."""
        T, H = x.shape
        k = topk_idx.shape[1]
        if H != self.H:
            raise ValueError("x's hidden size differs from the weights'")
        ws = workspace
        if ws is None or (ws.shape.T, ws.shape.H, ws.shape.I, ws.shape.E, ws.shape.k) != (T, H, self.I, self.E, k):
            ws = MoEWorkspace(T, H, self.I, self.E, k, device=x.device)
        ws.generation += 1  # the FP8 forward overwrites the saved activations
        idx = (topk_idx if topk_idx.dtype == torch.int32 else topk_idx.to(torch.int32)).contiguous()
        w = topk_weights.to(torch.float32).contiguous()
        xq = torch.empty(T, H, dtype=torch.uint8, device=x.device)
        xsf = torch.empty(T, H // 32, dtype=torch.uint8, device=x.device)
        y = torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
        with torch.cuda.device(x.device):
            B.moe_quantize_fp8(ws.shape, x.contiguous(), xq, xsf)
            B.moe_route_prologue(ws.shape, idx, ws.route)
            B.moe_forward_fp8(ws.shape, xq, xsf, self.W1_fp8, self.W1_sf, self.W2_fp8, self.W2_sf, w, ws.route,
                              ws.saved, y)
        return y

    __call__ = forward


def _nowhere():
    """The address of a weight that is not there."""


class DecodeLayer:
    """The whole expert layer for the few tokens of decoding (up to 64, k times
    which up to 1024): router, top-k and softmax, routed experts, shared expert and
    their sum, from the bf16 weights of training, in two kernels.

    router bf16 [H, E] (None: the routing is given to each call); W1 bf16 [E, H, 2I]
    (gate | up) and W2 bf16 [E, I, H] as ``moe_layer``'s; S1 [H, 2 Is] and S2 [Is, H]
    a shared expert, or None.  H, I and Is multiples of 8.  Keeps the weights as they
    are (contiguous ones are not copied; one whose storage the caller has freed is
    refused, and read where it lies once it is there again, as large as before).
    activation_clamp as in ``moe_layer``, for both kinds of experts.  Not
    differentiable."""

    def __init__(self, router, W1, W2, k: int, S1=None, S2=None, activation_clamp: float = 0.0):
        E, H, I2 = W1.shape
        I = I2 // 2
        if I2 % 2 or tuple(W2.shape) != (E, I, H):
            raise ValueError("expected W1 [E,H,2I], W2 [E,I,H]")
        if router is not None and tuple(router.shape) != (H, E):
            raise ValueError(f"expected router [{H}, {E}], got {list(router.shape)}")
        if (S1 is None) != (S2 is None):
            raise ValueError("a shared expert needs both S1 and S2")
        Is = 0 if S1 is None else S2.shape[0]
        if S1 is not None and (tuple(S1.shape) != (H, 2 * Is) or tuple(S2.shape) != (Is, H) or Is < 1):
            raise ValueError(f"expected S1 [{H}, 2 Is], S2 [Is, {H}], got {list(S1.shape)} and {list(S2.shape)}")
        weights = [router, W1, W2, S1, S2]
        for n, t in zip(("router", "W1", "W2", "S1", "S2"), weights):
            if t is None:
                continue
            if t.dtype != torch.bfloat16 or not t.is_cuda:
                raise TypeError(f"{n} must be a bfloat16 CUDA tensor")
            if t.get_device() != W1.get_device():
                raise ValueError(f"{n} is on {t.device}, W1 on {W1.device}")
        self._weights = tuple(None if t is None else t.detach().contiguous() for t in weights)
        self.E, self.H, self.I, self.k, self.Is = E, H, I, int(k), Is
        self.activation_clamp = float(activation_clamp)
        self.device = W1.get_device()
        self._sizes = {}  # T -> shape, reference to it, workspace bytes
        self._size(1)  # sizes that the kernels do not take are refused here
        self._where = [_nowhere if t is None else t.data_ptr for t in self._weights]
        self._addresses()

    def _addresses(self):
        """Where the weights are now.  Their storages are the caller's, who may free one and make
        it again between calls (sharded training does)."""
        at = [f() for f in self._where]
        if 0 in at:
            n = ("router", "W1", "W2", "S1", "S2")[at.index(0)]
            raise RuntimeError(f"the storage of {n} has been freed since the layer was made")
        return at

    # Read-only: their shapes and types are checked once, above.
    router = property(lambda self: self._weights[0])
    W1 = property(lambda self: self._weights[1])
    W2 = property(lambda self: self._weights[2])
    S1 = property(lambda self: self._weights[3])
    S2 = property(lambda self: self._weights[4])

    def _size(self, T):
        if T not in self._sizes:
            if T > B.DECODE_MAX_T or T * self.k > B.DECODE_MAX_SLOTS:
                raise ValueError(f"a decoding layer takes up to {B.DECODE_MAX_T} tokens with {B.DECODE_MAX_SLOTS} picks in "
                                 f"all, got {T} with {self.k} each (moe_layer takes more)")
            s = B.MoeDecodeShape(T, self.H, self.I, self.E, self.k, self.Is, self.activation_clamp)
            self._sizes[T] = (s, ctypes.byref(s), max(B.moe_decode_workspace(s), 16))
        return self._sizes[T]

    def forward(self, x, topk_idx=None, topk_w=None, out=None, return_routing: bool = False):
        """y bf16 [T, H] for x bf16 [T, H]; with return_routing (y, topk_idx int32
        [T, k], topk_w f32 [T, k]).  topk_idx int [T, k] and topk_w float [T, k]: the
        routing, of a layer without a router (ids outside the experts count for
        nothing)."""
        sh = x.shape
        if len(sh) != 2 or sh[1] != self.H:
            raise ValueError(f"expected x [T, {self.H}], got {list(sh)}")
        T, dev = sh[0], self.device
        s, ref, size = self._sizes.get(T) or self._size(T)
        weights = self._addresses()
        if (topk_idx is None and topk_w is None and out is None and weights[0] is not None and x.dtype is torch.bfloat16
                and x.get_device() == dev and dev == torch.cuda.current_device() and x.is_contiguous()):
            where = x.device
            y = torch.empty_like(x)
            if return_routing:
                topk_idx = torch.empty((T, self.k), dtype=torch.int32, device=where)
                topk_w = torch.empty((T, self.k), dtype=torch.float32, device=where)
                ws = torch.empty((size,), dtype=torch.uint8, device=where)
                at = ws.data_ptr()
                idx_at, w_at = topk_idx.data_ptr(), topk_w.data_ptr()
            else:  # behind the scratch: an allocation costs as much as a tenth of a small layer
                picks = 4 * T * self.k
                ws = torch.empty((size + 2 * picks,), dtype=torch.uint8, device=where)
                at = ws.data_ptr()
                idx_at, w_at = at + size, at + size + picks
            rc = B.lib().moe_decode_forward(ref, x.data_ptr(), *weights, idx_at, w_at, at, y.data_ptr(),
                                            torch._C._cuda_getCurrentRawStream(dev))
            if rc:
                B._check(rc)
            return (y, topk_idx, topk_w) if return_routing else y
        if self.router is None:
            if topk_idx is None or topk_w is None or topk_idx.shape != (T, self.k) or topk_w.shape != (T, self.k):
                raise ValueError(f"a layer without a router needs topk_idx and topk_w [{T}, {self.k}]")
            topk_idx, topk_w = _expert_ids(topk_idx, self.E).contiguous(), topk_w.to(torch.float32).contiguous()
        elif topk_idx is not None or topk_w is not None:
            raise ValueError("this layer has a router of its own")
        with _on_device(x, dev):
            if self.router is not None:
                topk_idx = torch.empty((T, self.k), dtype=torch.int32, device=x.device)
                topk_w = torch.empty((T, self.k), dtype=torch.float32, device=x.device)
            ws = torch.empty((size,), dtype=torch.uint8, device=x.device)
            y = torch.empty((T, self.H), dtype=torch.bfloat16, device=x.device) if out is None else out
            B.moe_decode_forward(s, x if x.is_contiguous() else x.contiguous(), *self._weights, topk_idx, topk_w, ws, y)
        return (y, topk_idx, topk_w) if return_routing else y

    __call__ = forward


def _expert_ids(topk_idx, E):
    """Expert ids of any integer type as int32; what lies outside [0, E) stays outside."""
    if topk_idx.dtype is torch.int32:
        return topk_idx
    if topk_idx.is_floating_point() or topk_idx.is_complex():
        raise TypeError(f"topk_idx must be of an integer type, got {topk_idx.dtype}")
    # in 64 bits: a narrow type holds neither bound, and 32 bits would cut a wide id to an expert's
    return topk_idx.to(torch.int64).clamp(-1, E).to(torch.int32)


def _on_device(x, dev):
    """Context in which device dev, where x has to be, is current."""
    if x.get_device() != dev:
        if not x.is_cuda:
            raise TypeError("x must be a CUDA tensor")
        raise ValueError(f"x is on {x.device}, the weights on cuda:{dev}")
    return contextlib.nullcontext() if dev == torch.cuda.current_device() else torch.cuda.device(dev)


def train_step_from_host(x_h, topk_idx_h, topk_w_h, dY_h, W1, W2, ws: MoEWorkspace, outs: dict):
    """One forward+backward of the layer fed from pinned HOST buffers.

    Copies x, topk_idx, topk_weights and dY host->device, runs the routing
    prologue, forward and backward through the C ABI, and copies y, dx and
    d(topk_weights) back to pinned host buffers (outs['y_h'], outs['dx_h'],
    outs['dw_h']).  The weight gradients stay on the device (outs['dW1'],
    outs['dW2']) where an optimizer would consume them.  All on the current
    stream; returns without synchronising."""
    s = ws.shape
    x = outs["x"]
    x.copy_(x_h, non_blocking=True)
    outs["idx"].copy_(topk_idx_h, non_blocking=True)
    outs["w"].copy_(topk_w_h, non_blocking=True)
    outs["dY"].copy_(dY_h, non_blocking=True)
    B.moe_route_prologue(s, outs["idx"], ws.route)
    B.moe_forward(s, x, W1, W2, outs["w"], ws.route, ws.saved, outs["y"])
    B.moe_backward(s, outs["dY"], x, W1, W2, outs["w"], ws.route, ws.saved, ws.bwd, outs["dx"], outs["dW1"],
                   outs["dW2"], outs["dw"])
    outs["y_h"].copy_(outs["y"], non_blocking=True)
    outs["dx_h"].copy_(outs["dx"], non_blocking=True)
    outs["dw_h"].copy_(outs["dw"], non_blocking=True)


class HostPipeline:
    """Forward+backward steps fed from pinned HOST buffers, with the copies
    overlapped with the layer's kernels.

    ``submit(x_h, topk_idx_h, topk_w_h, dY_h, y_h, dx_h, dw_h)`` enqueues one
    step and returns at once: the host->device copies of the step's inputs go
    on an upload stream, the routing prologue, forward and backward on the
    compute stream (the current stream when the pipeline was made), and the
    device->host copies of y (as soon as the forward is done) and of dx and
    d(topk_weights) (after the backward) on a download stream.  Inputs and
    outputs on the device are double-buffered, so step n+1's uploads run
    during step n's kernels and step n's downloads during step n+1's.  The
    weight gradients stay on the device in ``dW1``/``dW2`` (overwritten by
    every step), where an optimizer would consume them.  Host buffers handed
    to ``submit`` must stay untouched until ``synchronize()``."""

    def __init__(self, ws: MoEWorkspace, W1, W2, dW1=None, dW2=None):
        s = ws.shape
        dev = ws.device
        self.ws, self.W1, self.W2 = ws, W1, W2
        self.compute = torch.cuda.current_stream(dev)
        self.up = torch.cuda.Stream(dev)
        self.down = torch.cuda.Stream(dev)
        bf = torch.bfloat16

        def slot():
            return dict(x=torch.empty(s.T, s.H, dtype=bf, device=dev),
                        idx=torch.empty(s.T, s.k, dtype=torch.int32, device=dev),
                        w=torch.empty(s.T, s.k, dtype=torch.float32, device=dev),
                        dY=torch.empty(s.T, s.H, dtype=bf, device=dev),
                        y=torch.empty(s.T, s.H, dtype=bf, device=dev),
                        dx=torch.empty(s.T, s.H, dtype=bf, device=dev),
                        dw=torch.empty(s.T, s.k, dtype=torch.float32, device=dev),
                        uploaded=torch.cuda.Event(), fwd_done=torch.cuda.Event(), bwd_done=torch.cuda.Event(),
                        downloaded=torch.cuda.Event(), used=False)

        self.slots = [slot(), slot()]
        self.dW1 = torch.empty_like(W1) if dW1 is None else dW1
        self.dW2 = torch.empty_like(W2) if dW2 is None else dW2
        self.n = 0

    def submit(self, x_h, topk_idx_h, topk_w_h, dY_h, y_h, dx_h, dw_h):
        sl = self.slots[self.n % 2]
        self.n += 1
        s = self.ws.shape
        if sl["used"]:
            # the slot's previous step must be done with its inputs and
            # outputs before they are overwritten
            self.up.wait_event(sl["bwd_done"])
            self.up.wait_event(sl["downloaded"])
        sl["used"] = True
        with torch.cuda.stream(self.up):
            sl["x"].copy_(x_h, non_blocking=True)
            sl["idx"].copy_(topk_idx_h, non_blocking=True)
            sl["w"].copy_(topk_w_h, non_blocking=True)
            sl["dY"].copy_(dY_h, non_blocking=True)
            sl["uploaded"].record(self.up)
        c = self.compute
        c.wait_event(sl["uploaded"])
        B.moe_route_prologue(s, sl["idx"], self.ws.route, stream=c)
        B.moe_forward(s, sl["x"], self.W1, self.W2, sl["w"], self.ws.route, self.ws.saved, sl["y"], stream=c)
        sl["fwd_done"].record(c)
        B.moe_backward(s, sl["dY"], sl["x"], self.W1, self.W2, sl["w"], self.ws.route, self.ws.saved, self.ws.bwd,
                       sl["dx"], self.dW1, self.dW2, sl["dw"], stream=c)
        sl["bwd_done"].record(c)
        with torch.cuda.stream(self.down):
            self.down.wait_event(sl["fwd_done"])
            y_h.copy_(sl["y"], non_blocking=True)
            self.down.wait_event(sl["bwd_done"])
            dx_h.copy_(sl["dx"], non_blocking=True)
            dw_h.copy_(sl["dw"], non_blocking=True)
            sl["downloaded"].record(self.down)

    def synchronize(self):
        """Makes the compute stream wait for every copy enqueued so far."""
        self.compute.wait_stream(self.up)
        self.compute.wait_stream(self.down)
