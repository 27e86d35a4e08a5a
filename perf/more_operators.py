"""Cases of the operators that complete a block around the routed experts: the
joint between two halves of a block, its projections, and the whole expert
layer for the few tokens of decoding.

  joint   s = alpha residual + gate u,  u = norm(out) post_weight + post_bias (or out),
          n = norm(s) weight + bias, and the backward pass of both outputs
          (dout, dresidual, dweight, dbias, dpost_weight, dpost_bias, dgate)
  linear  y = act(x W + bias) + residual, and its backward pass
          (dx, dW, dbias; the residual's gradient is dy)
  decode  router logits x R, the k largest (equal ones: the lower id), softmax
          over them, the gated experts' weighted sum, plus a shared expert

norm is a layer norm or, without mean and usually without bias, an RMS norm;
act is silu, gelu (with erf), gelu_tanh or nothing.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # the joint of a training step: the smallest layer with everything switched on, the V2-Lite-shaped one in
        # its commonest form (residual sum and RMS norm), the V3-shaped one with norms before and after and a gate per token
        {"name": "joint_step_64x128_f32", "op": "joint", "dir": "step", "rows": 64, "H": 128, "type": "f32", "kind": "layer",
         "bias": True, "post": True, "gate": "channel", "alpha": 0.5},
        {"name": "joint_step_4096x2048", "op": "joint", "dir": "step", "rows": 4096, "H": 2048, "type": "bf16", "kind": "rms",
         "bias": False, "post": False, "gate": "none", "alpha": 1.0},
        {"name": "joint_step_8192x7168", "op": "joint", "dir": "step", "rows": 8192, "H": 7168, "type": "bf16", "kind": "rms",
         "bias": False, "post": True, "gate": "token", "alpha": 1.0},
        # the joint of a serving batch with a width that no vector divides
        {"name": "joint_fwd_777x1001_f16", "op": "joint", "dir": "fwd", "rows": 777, "H": 1001, "type": "f16", "kind": "layer",
         "bias": True, "post": True, "gate": "channel", "alpha": 1.25},
        # projections: one of a few decoding sequences; training steps of an odd small layer, a V2-Lite-shaped one with an
        # activation, and one into the V3-shaped residual stream
        {"name": "linear_fwd_8x2048x7168", "op": "linear", "dir": "fwd", "T": 8, "K": 2048, "N": 7168, "act": "none",
         "bias": True, "residual": True},
        {"name": "linear_step_777x1160x712", "op": "linear", "dir": "step", "T": 777, "K": 1160, "N": 712, "act": "gelu",
         "bias": True, "residual": True},
        {"name": "linear_step_4096x2048x2816", "op": "linear", "dir": "step", "T": 4096, "K": 2048, "N": 2816, "act": "silu",
         "bias": True, "residual": False},
        {"name": "linear_step_8192x2048x7168", "op": "linear", "dir": "step", "T": 8192, "K": 2048, "N": 7168, "act": "none",
         "bias": True, "residual": True},
        # the expert layer of decoding: a handful of tokens of the smallest layer, one V3-shaped token, a V2-Lite-shaped
        # batch with its shared expert, a V3-shaped batch
        {"name": "decode_4_tiny", "op": "decode", "T": 4, "H": 128, "I": 64, "E": 8, "k": 2, "shared": 0},
        {"name": "decode_1_v3", "op": "decode", "T": 1, "H": 7168, "I": 2048, "E": 256, "k": 8, "shared": 0},
        {"name": "decode_32_v2lite_shared", "op": "decode", "T": 32, "H": 2048, "I": 1408, "E": 64, "k": 6, "shared": 2816},
        {"name": "decode_16_v3_shared", "op": "decode", "T": 16, "H": 7168, "I": 2048, "E": 256, "k": 8, "shared": 2048},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(("joint", "linear", "decode"))
    if op == "joint":
        return {"op": op, "dir": rng.choice(("step", "step", "fwd")), "rows": _log(rng, 1, 8192), "H": _log(rng, 64, 7168),
                "type": rng.choice(("bf16", "bf16", "f16", "f32")), "kind": rng.choice(("layer", "rms")),
                "bias": rng.random() < 0.5, "post": rng.random() < 0.5, "gate": rng.choice(("none", "channel", "token")),
                "alpha": rng.choice((1.0, 1.0, 0.5, 1.25))}
    if op == "linear":
        K, N, step = _log(rng, 64, 7168, 8), _log(rng, 64, 7168, 8), rng.random() < 0.7
        T = _log(rng, 16, 8192) if step else _log(rng, 1, 512)
        return {"op": op, "dir": "step" if step else "fwd", "T": min(T, 8192 * 2048 * 7168 // (K * N)), "K": K, "N": N,
                "act": rng.choice(("none", "silu", "gelu", "gelu_tanh")), "bias": rng.random() < 0.7,
                "residual": rng.random() < 0.5}
    H, I, E, k = _log(rng, 64, 4096, 8), _log(rng, 32, 1408, 8), rng.choice((8, 16, 60, 64, 101, 160)), rng.randint(1, 8)
    T = max(1, min(_log(rng, 1, 64), 128 * 7168 * 2048 // (k * H * I)))
    return {"op": op, "T": T, "H": H, "I": I, "E": E, "k": k, "shared": rng.choice((0, I, 2 * I))}


# ------------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + salt)
    return g


def _randn(shape, std, dtype, g):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _experts(E, rows, cols, g):
    """bf16 [E, rows, cols] of standard deviation rows^-0.5: the sum of four uniform numbers, drawn as the 16-bit
    parts of whole numbers, an expert at a time at most."""
    out = torch.empty((E, rows, cols), dtype=BF16, device="cuda")
    n, std = rows * cols, (rows * 4 * (2.0 ** 32 - 1) / 12.0) ** 0.5
    per = max(1, (1 << 26) // n)
    for e in range(0, E, per):
        m = min(per, E - e)
        parts = torch.empty(m * n, dtype=torch.int64, device="cuda").random_(-2 ** 63, None, generator=g).view(torch.int16)
        out[e:e + m] = (parts.view(m, rows, cols, 4).sum(dim=3, dtype=F32).add_(2.0).mul_(1.0 / std)).to(BF16)
    return out


def prepare(case, seed):
    g, op = _gen(seed, 1), case["op"]
    s = {"case": case}
    if op == "joint":
        rows, H, t = case["rows"], case["H"], TYPES[case["type"]]
        # a residual stream: rows of different scale with an offset, a few strong channels; a block's output beside it
        r = torch.randn((rows, H), generator=g, device="cuda")
        r[:, :: max(1, H // 4)] *= 8.0
        r = r * (0.5 + torch.rand((rows, 1), generator=g, device="cuda")) + 0.3 * torch.randn((rows, 1), generator=g, device="cuda")
        s["residual"], s["out"] = r.to(t), _randn((rows, H), 0.7, t, g)
        s["weight"] = 1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")
        s["bias"] = 0.1 * torch.randn(H, generator=g, device="cuda") if case["bias"] else None
        s["post_weight"] = 1.0 + 0.2 * torch.randn(H, generator=g, device="cuda") if case["post"] else None
        s["post_bias"] = 0.1 * torch.randn(H, generator=g, device="cuda") if case["post"] and case["bias"] else None
        s["gate"] = {"none": None, "channel": 0.5 + 0.2 * torch.randn(H, generator=g, device="cuda"),
                     "token": torch.sigmoid(torch.randn((rows, 1), generator=g, device="cuda"))}[case["gate"]]
        s["eps"] = 1e-5
        if case["dir"] == "step":
            s["dstream"], s["dnormed"] = _randn((rows, H), 1.0, t, g), _randn((rows, H), 1.0, t, g)
        return s
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        s["x"] = _randn((T, K), 1.0, BF16, g)
        s["W"] = _randn((K, N), K ** -0.5, BF16, g)
        s["bias"] = _randn((N,), 0.5, BF16, g) if case["bias"] else None
        s["residual"] = _randn((T, N), 1.0, BF16, g) if case["residual"] else None
        s["act"] = None if case["act"] == "none" else case["act"]
        if case["dir"] == "step":
            s["dy"] = _randn((T, N), 1.0, BF16, g)
        return s
    T, H, I, E, k, shared = (case[n] for n in ("T", "H", "I", "E", "k", "shared"))
    s["x"] = _randn((T, H), 1.0, BF16, g)
    s["router"] = _randn((H, E), H ** -0.5, BF16, g)
    s["W1"], s["W2"] = _experts(E, H, 2 * I, g), _experts(E, I, H, g)
    s["S1"] = _randn((H, 2 * shared), H ** -0.5, BF16, g) if shared else None
    s["S2"] = _randn((shared, H), shared ** -0.5, BF16, g) if shared else None
    if own:  # a serving program makes the layer once and keeps it
        from routed_grouped_gemm_routing_gb300.layer import DecodeLayer

        s["layer"] = DecodeLayer(s["router"], s["W1"], s["W2"], k, s["S1"], s["S2"])
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"joint": _own_joint, "linear": _own_linear, "decode": _own_decode}[op](s)
    return {"joint": _plain_joint, "linear": _plain_linear, "decode": _plain_decode}[op](s)


def _own_joint(s):
    from routed_grouped_gemm_routing_gb300.block import residual_norm_backward, residual_norm_forward

    alpha, kind = s["case"]["alpha"], s["case"]["kind"]
    stream, normed, stats = residual_norm_forward(
        s["out"], s["residual"], s["weight"], bias=s["bias"], post_weight=s["post_weight"], post_bias=s["post_bias"],
        gate=s["gate"], residual_scale=alpha, eps=s["eps"], kind=kind)
    if "dstream" not in s:
        return {"stream": stream, "normed": normed}
    grads = residual_norm_backward(
        s["dstream"], s["dnormed"], s["out"], s["residual"], s["weight"], stats, bias=s["bias"],
        post_weight=s["post_weight"], post_bias=s["post_bias"], gate=s["gate"], residual_scale=alpha, kind=kind)
    names = ("dout", "dresidual", "dweight", "dbias", "dpost_weight", "dpost_bias", "dgate")
    return {"stream": stream, "normed": normed, **{n: v for n, v in zip(names, grads) if v is not None}}


def _own_linear(s):
    from routed_grouped_gemm_routing_gb300.block import linear_backward, linear_forward

    step = "dy" in s
    y, z = linear_forward(s["x"], s["W"], bias=s["bias"], residual=s["residual"], activation=s["act"], for_backward=step)
    if not step:
        return {"y": y}
    dx, dW, db = linear_backward(s["dy"], s["x"], s["W"], z, bias=s["bias"], activation=s["act"])
    return {"y": y, "dx": dx, "dW": dW, **({"dbias": db} if db is not None else {})}


def _own_decode(s):
    y, idx, w = s["layer"](s["x"], return_routing=True)
    return {"y": y, "topk_idx": idx, "topk_w": w}


def _plain_stats(v, kind, eps):
    """(v about its mean, 1 / its root mean square) per row."""
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    return v, (v.square().mean(dim=1, keepdim=True) + eps).rsqrt()


def _plain_norm_grad(d, z, rstd, kind):
    """The gradient through z = (v - mean) rstd."""
    d0 = d - d.mean(dim=1, keepdim=True) if kind == "layer" else d
    return rstd * (d0 - z * (d * z).mean(dim=1, keepdim=True))


def _plain_joint(s):
    t, kind, eps, alpha = s["out"].dtype, s["case"]["kind"], s["eps"], s["case"]["alpha"]
    u = out = s["out"].to(F32)
    if s["post_weight"] is not None:
        oc, orstd = _plain_stats(out, kind, eps)
        oz = oc * orstd
        u = oz * s["post_weight"]
        if s["post_bias"] is not None:
            u = u + s["post_bias"]
    gated = u if s["gate"] is None else u * s["gate"]
    stream = s["residual"].to(F32) * alpha + gated
    sc, rstd = _plain_stats(stream, kind, eps)
    z = sc * rstd
    n = z * s["weight"]
    if s["bias"] is not None:
        n = n + s["bias"]
    result = {"stream": stream.to(t), "normed": n.to(t)}
    if "dstream" not in s:
        return result
    dn = s["dnormed"].to(F32)
    ds = s["dstream"].to(F32) + _plain_norm_grad(dn * s["weight"], z, rstd, kind)
    du = ds if s["gate"] is None else ds * s["gate"]
    dout = du if s["post_weight"] is None else _plain_norm_grad(du * s["post_weight"], oz, orstd, kind)
    result |= {"dout": dout.to(t), "dresidual": (ds * alpha).to(t), "dweight": (dn * z).sum(dim=0)}
    if s["bias"] is not None:
        result["dbias"] = dn.sum(dim=0)
    if s["post_weight"] is not None:
        result["dpost_weight"] = (du * oz).sum(dim=0)
        if s["post_bias"] is not None:
            result["dpost_bias"] = du.sum(dim=0)
    if s["gate"] is not None:
        result["dgate"] = (ds * u).sum(dim=0) if s["case"]["gate"] == "channel" else (ds * u).sum(dim=1, keepdim=True)
    return result


def _plain_act(z, act):
    """(act(z), act'(z))."""
    if act is None:
        return z, torch.ones_like(z)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5))
        return z * p, p + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    c = (2.0 / math.pi) ** 0.5
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _plain_linear(s):
    x, W = s["x"].to(F32), s["W"].to(F32)
    z = x @ W
    if s["bias"] is not None:
        z = z + s["bias"].to(F32)
    y, slope = _plain_act(z, s["act"])
    if s["residual"] is not None:
        y = y + s["residual"].to(F32)
    if "dy" not in s:
        return {"y": y.to(BF16)}
    dz = s["dy"].to(F32) * slope
    return {"y": y.to(BF16), "dx": (dz @ W.t()).to(BF16), "dW": (x.t() @ dz).to(BF16),
            **({"dbias": dz.sum(dim=0).to(BF16)} if s["bias"] is not None else {})}


def _plain_gated(x, W1, W2):
    """(silu(x W1[.., :I]) * (x W1[.., I:])) W2, batched where the weights are."""
    h = x @ W1
    I = W2.shape[-2]
    a = h[..., :I] / (1.0 + torch.exp(-h[..., :I])) * h[..., I:]
    return a @ W2


def _plain_decode(s):
    case = s["case"]
    T, H, k = case["T"], case["H"], case["k"]
    x = s["x"].to(F32)
    # which experts a token takes is a border: the logits in 64 bits, equal ones in the order of their ids
    logits, order = torch.sort(s["x"].to(F64) @ s["router"].to(F64), dim=1, descending=True, stable=True)
    idx, chosen = order[:, :k], logits[:, :k]
    e = torch.exp(chosen - chosen[:, :1])
    w = (e / e.sum(dim=1, keepdim=True)).to(F32)
    slots = idx.reshape(-1)
    o = _plain_gated(x.repeat_interleave(k, dim=0).unsqueeze(1), s["W1"][slots].to(F32), s["W2"][slots].to(F32))
    y = (o.view(T, k, H) * w.unsqueeze(2)).sum(dim=1)
    if s["S1"] is not None:
        y = y + _plain_gated(x, s["S1"].to(F32), s["S2"].to(F32))
    return {"y": y.to(BF16), "topk_idx": idx.to(torch.int32), "topk_w": w}


# ------------------------------------------------------- floors and 64 bits
def work(case):
    op = case["op"]
    if op == "joint":
        n, es = case["rows"] * case["H"], 4 if case["type"] == "f32" else 2
        step = case["dir"] == "step"
        params = 4 * case["H"] * (1 + case["bias"] + case["post"] * (1 + case["bias"]) + (case["gate"] == "channel"))
        return {"bytes": n * es * (8 if step else 4) + params * (2 if step else 1), "flops": n * (50 if step else 20)}
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        step, res = case["dir"] == "step", case["residual"]
        fwd = T * K + K * N + T * N * (2 if res else 1)
        return {"bytes": 2 * (fwd + (T * N + T * K + K * N if step else 0)), "flops": (6 if step else 2) * T * K * N}
    T, H, I, E, k, shared = (case[n] for n in ("T", "H", "I", "E", "k", "shared"))
    used = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token picks, each read once
    return {"bytes": 2 * (used * 3 * H * I + 3 * H * shared + H * E + 2 * T * H) + 8 * T * k,
            "flops": 6 * T * H * (k * I + shared) + 2 * T * H * E}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"joint": _exact_joint, "linear": _exact_linear, "decode": _exact_decode}[case["op"]](s)


def _exact_joint(s):
    """By autograd in 64 bits, from the definition."""
    names = ("out", "residual", "weight", "bias", "post_weight", "post_bias", "gate")
    v = {n: None if s[n] is None else s[n].double().requires_grad_() for n in names}

    def norm(a, weight, bias):
        mean = a.mean(1, True) if s["case"]["kind"] == "layer" else 0.0
        a = (a - mean) / torch.sqrt(torch.mean((a - mean) ** 2, 1, True) + s["eps"]) * weight
        return a if bias is None else a + bias

    u = v["out"] if v["post_weight"] is None else norm(v["out"], v["post_weight"], v["post_bias"])
    stream = s["case"]["alpha"] * v["residual"] + (u if v["gate"] is None else v["gate"] * u)
    normed = norm(stream, v["weight"], v["bias"])
    result = {"stream": stream.detach(), "normed": normed.detach()}
    if "dstream" in s:
        wanted = [n for n in names if v[n] is not None]
        grads = torch.autograd.grad((stream, normed), [v[n] for n in wanted], (s["dstream"].double(), s["dnormed"].double()))
        result |= {"d" + n: d for n, d in zip(wanted, grads)}
    return result


def _exact_linear(s):
    x, W = s["x"].double(), s["W"].double()
    z = torch.einsum("tk,kn->tn", x, W) + (0.0 if s["bias"] is None else s["bias"].double())
    z.requires_grad_()
    f = {None: lambda v: v * 1.0, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[s["act"]]
    a = f(z)
    result = {"y": a.detach() + (0.0 if s["residual"] is None else s["residual"].double())}
    if "dy" in s:
        dz, = torch.autograd.grad(a, z, s["dy"].double())
        result |= {"dx": torch.einsum("tn,kn->tk", dz, W), "dW": torch.einsum("tk,tn->kn", x, dz)}
        if s["bias"] is not None:
            result["dbias"] = torch.einsum("tn->n", dz)
    return result


def _exact_decode(s):
    x, k, T = s["x"].double(), s["case"]["k"], s["case"]["T"]
    logits = torch.einsum("th,he->te", x, s["router"].double())
    idx = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    w = torch.softmax(torch.gather(logits, 1, idx), dim=1)

    def expert(v, W1, W2):
        g, u = (v @ W1.double()).chunk(2, dim=1)
        return (torch.nn.functional.silu(g) * u) @ W2.double()

    y = torch.zeros((T, s["case"]["H"]), dtype=F64, device="cuda") if s["S1"] is None else expert(x, s["S1"], s["S2"])
    for e in torch.unique(idx).tolist():
        t, j = torch.nonzero(idx == e, as_tuple=True)
        y.index_add_(0, t, expert(x[t], s["W1"][e], s["W2"][e]) * w[t, j][:, None])
    return {"y": y, "topk_idx": idx.to(torch.int32), "topk_w": w}
