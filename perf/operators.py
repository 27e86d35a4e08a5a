"""Cases of the operators that stand beside the routed experts in a block:
layer norm in front of router and experts, the dense gated feed-forward block
(the shared expert), and products with 4-bit weights for serving.

  norm    y = (x - mean) * rstd * weight + bias over the last axis, and its
          backward pass (dx, dweight, dbias)
  ffn     y = (silu(x W1[:, :I]) * (x W1[:, I:])) W2, and its backward pass
          (dx, dW1, dW2)
  matvec  y = x W^T with W held as 4-bit codes and one scale per group
  experts the routed experts (top-k, weighted sum) with both weights of every
          expert held that way

A 4-bit weight of value (code - 8) * scale: row n of the matrix has K codes,
128 of them in 64 bytes, that is in 16 little-endian words; word 4 t + j holds
the eight codes 32 j + 8 t .. + 7, code 2 m of them in nibble m and code
2 m + 1 in nibble m + 4.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # the norm of a training step: the smallest layer, the V2-Lite-shaped and the V3-shaped one
        {"name": "norm_step_64x128_f32", "op": "norm", "dir": "step", "rows": 64, "H": 128, "type": "f32", "bias": True},
        {"name": "norm_step_4096x2048", "op": "norm", "dir": "step", "rows": 4096, "H": 2048, "type": "bf16", "bias": True},
        {"name": "norm_step_8192x7168", "op": "norm", "dir": "step", "rows": 8192, "H": 7168, "type": "bf16", "bias": True},
        # the norm of a serving batch with a width that no vector divides
        {"name": "norm_fwd_777x1001_f16", "op": "norm", "dir": "fwd", "rows": 777, "H": 1001, "type": "f16", "bias": False},
        # the shared expert: a few decoding sequences; training steps of an odd
        # small layer, of the V2-Lite-shaped and of the V3-shaped one
        {"name": "ffn_fwd_8x2048x1408", "op": "ffn", "dir": "fwd", "T": 8, "H": 2048, "I": 1408},
        {"name": "ffn_step_777x1160x712", "op": "ffn", "dir": "step", "T": 777, "H": 1160, "I": 712},
        {"name": "ffn_step_4096x2048x1408", "op": "ffn", "dir": "step", "T": 4096, "H": 2048, "I": 1408},
        {"name": "ffn_step_8192x7168x2048", "op": "ffn", "dir": "step", "T": 8192, "H": 7168, "I": 2048},
        # one projection for one token, and for a batch of 12 with a ragged output
        {"name": "matvec_1_7168x2048_g128", "op": "matvec", "T": 1, "N": 7168, "K": 2048, "group": 128},
        {"name": "matvec_12_16380x7168_g32", "op": "matvec", "T": 12, "N": 16380, "K": 7168, "group": 32},
        # the routed experts of one decoded token (V3-shaped), and of a batch of 32 (V2-Lite-shaped)
        {"name": "experts_1_v3_g128", "op": "experts", "T": 1, "H": 7168, "I": 2048, "E": 256, "k": 8, "group": 128},
        {"name": "experts_32_v2lite_g64", "op": "experts", "T": 32, "H": 2048, "I": 1408, "E": 64, "k": 6, "group": 64},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(("norm", "ffn", "matvec", "experts"))
    if op == "norm":
        return {"op": op, "dir": rng.choice(("step", "step", "fwd")), "rows": _log(rng, 1, 8192), "H": _log(rng, 64, 7168),
                "type": rng.choice(("bf16", "bf16", "f16", "f32")), "bias": rng.random() < 0.7}
    if op == "ffn":
        if rng.random() < 0.3:
            return {"op": op, "dir": "fwd", "T": _log(rng, 1, 512), "H": _log(rng, 128, 7168, 8), "I": _log(rng, 64, 2048, 8)}
        return {"op": op, "dir": "step", "T": _log(rng, 16, 8192), "H": _log(rng, 128, 7168, 8), "I": _log(rng, 64, 2048, 8)}
    if op == "matvec":
        return {"op": op, "T": _log(rng, 1, 32), "N": _log(rng, 64, 16384), "K": _log(rng, 128, 7168, 128),
                "group": rng.choice((32, 64, 128))}
    E = rng.choice((8, 16, 60, 64, 101, 160))
    return {"op": op, "T": _log(rng, 1, 32), "H": _log(rng, 256, 4096, 128), "I": _log(rng, 128, 1408, 128), "E": E,
            "k": rng.randint(1, 8), "group": rng.choice((32, 64, 128))}


# ------------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + salt)
    return g


def _randn(shape, std, dtype, g):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _codes(rows, K, g):
    """uint8 [rows, K / 2]: codes 1..15 around 8, the sum of two uniform draws (as the weights of a group
    scaled to their largest are spread)."""
    n = rows * K // 16
    a = torch.empty(n, dtype=torch.int64, device="cuda").random_(generator=g)
    b = torch.empty(n, dtype=torch.int64, device="cuda").random_(generator=g)
    m = 0x7777777777777777
    a.bitwise_and_(m).add_(b.bitwise_and_(m)).add_(0x1111111111111111)
    return a.view(torch.uint8).view(rows, K // 2)


def _scales(rows, K, group, g):
    s = 0.5 + torch.rand((rows, K // group), generator=g, device="cuda")
    return (s / (3.24 * math.sqrt(K))).to(BF16)


def prepare(case, seed):
    g, op = _gen(seed, 1), case["op"]
    s = {"case": case}
    if op == "norm":
        rows, H, t = case["rows"], case["H"], TYPES[case["type"]]
        # activations of a residual stream: rows of different scale with an offset, a few strong channels
        x = torch.randn((rows, H), generator=g, device="cuda")
        x[:, :: max(1, H // 4)] *= 8.0
        x = x * (0.5 + torch.rand((rows, 1), generator=g, device="cuda")) + 0.3 * torch.randn((rows, 1), generator=g, device="cuda")
        s["x"] = x.to(t)
        s["weight"] = 1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")
        s["bias"] = 0.1 * torch.randn(H, generator=g, device="cuda") if case["bias"] else None
        s["eps"] = 1e-5
        if case["dir"] == "step":
            s["dy"] = _randn((rows, H), 1.0, t, g)
        return s
    if op == "ffn":
        T, H, I = case["T"], case["H"], case["I"]
        s["x"] = _randn((T, H), 1.0, BF16, g)
        s["W1"] = _randn((H, 2 * I), H ** -0.5, BF16, g)
        s["W2"] = _randn((I, H), I ** -0.5, BF16, g)
        if case["dir"] == "step":
            s["dy"] = _randn((T, H), 1.0, BF16, g)
        if own:  # buffers that a training program keeps from step to step
            from routed_grouped_gemm_routing_gb300.block import FFNWorkspace

            s["ws"] = FFNWorkspace(T, H, I)
        return s
    if op == "matvec":
        T, N, K, group = case["T"], case["N"], case["K"], case["group"]
        s["x"] = _randn((T, K), 1.0, BF16, g)
        s["q"], s["sf"] = _codes(N, K, g), _scales(N, K, group, g)
        if own:
            from routed_grouped_gemm_routing_gb300.block import W4Linear

            s["linear"] = W4Linear(s["q"], s["sf"], group)
        return s
    T, H, I, E, k, group = (case[n] for n in ("T", "H", "I", "E", "k", "group"))
    s["x"] = _randn((T, H), 1.0, BF16, g)
    s["W1_q"], s["W1_sf"] = _codes(E * 2 * I, H, g).view(E, 2 * I, H // 2), _scales(E * 2 * I, H, group, g).view(E, 2 * I, -1)
    s["W2_q"], s["W2_sf"] = _codes(E * H, I, g).view(E, H, I // 2), _scales(E * H, I, group, g).view(E, H, -1)
    w, idx = torch.topk(torch.randn((T, E), generator=g, device="cuda"), k, dim=1)
    s["topk_idx"], s["topk_w"] = idx.to(torch.int32), torch.softmax(w, dim=1)
    if own:
        from routed_grouped_gemm_routing_gb300.block import W4Experts

        s["experts"] = W4Experts(s["W1_q"], s["W1_sf"], s["W2_q"], s["W2_sf"], group)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return {"norm": _own_norm, "ffn": _own_ffn, "matvec": lambda v: v["linear"](v["x"]),
                "experts": lambda v: v["experts"](v["x"], v["topk_idx"], v["topk_w"])}[op](s)
    return {"norm": _plain_norm, "ffn": _plain_ffn, "matvec": _plain_matvec, "experts": _plain_experts}[op](s)


def _own_norm(s):
    from routed_grouped_gemm_routing_gb300.block import layer_norm_backward, layer_norm_forward

    y, mean, rstd = layer_norm_forward(s["x"], s["weight"], s["bias"], s["eps"])
    if "dy" not in s:
        return {"y": y}
    dx, dw, db = layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd, bias=s["bias"] is not None)
    return {"y": y, "dx": dx, "dweight": dw, **({"dbias": db} if db is not None else {})}


def _own_ffn(s):
    from routed_grouped_gemm_routing_gb300.block import ffn_backward, ffn_forward

    y = ffn_forward(s["x"], s["W1"], s["W2"], s["ws"])
    if "dy" not in s:
        return {"y": y}
    dx, dW1, dW2 = ffn_backward(s["dy"], s["x"], s["W1"], s["W2"], s["ws"])
    return {"y": y, "dx": dx, "dW1": dW1, "dW2": dW2}


def _plain_norm(s):
    t, w = s["x"].dtype, s["weight"]
    x = s["x"].to(F32)
    xc = x - x.mean(dim=1, keepdim=True)
    rstd = (xc.square().mean(dim=1, keepdim=True) + s["eps"]).rsqrt()
    xhat = xc * rstd
    y = xhat * w
    if s["bias"] is not None:
        y = y + s["bias"]
    if "dy" not in s:
        return {"y": y.to(t)}
    dy = s["dy"].to(F32)
    gr = dy * w
    dx = rstd * (gr - gr.mean(dim=1, keepdim=True) - xhat * (gr * xhat).mean(dim=1, keepdim=True))
    out = {"y": y.to(t), "dx": dx.to(t), "dweight": (dy * xhat).sum(dim=0)}
    if s["bias"] is not None:
        out["dbias"] = dy.sum(dim=0)
    return out


def _plain_ffn(s):
    I = s["case"]["I"]
    x, W1, W2 = s["x"].to(F32), s["W1"].to(F32), s["W2"].to(F32)
    h = x @ W1
    gate, up = h[:, :I], h[:, I:]
    sig = 1.0 / (1.0 + torch.exp(-gate))
    a = gate * sig * up
    y = (a @ W2).to(BF16)
    if "dy" not in s:
        return {"y": y}
    dy = s["dy"].to(F32)
    da = dy @ W2.t()
    dh = torch.cat((da * up * sig * (1.0 + gate * (1.0 - sig)), da * gate * sig), dim=1)
    return {"y": y, "dx": (dh @ W1.t()).to(BF16), "dW1": (x.t() @ dh).to(BF16), "dW2": (a.t() @ dy).to(BF16)}


def _plain_weights(q, sf, group):
    """float32 [..., K] of the codes [..., K / 2] and the scales [..., K / group]."""
    K = q.shape[-1] * 2
    words = q.contiguous().view(torch.int32).reshape(-1, K // 128, 4, 4, 1)  # row, block, t, j
    shift = torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)
    nib = (words >> shift) & 15  # nibble p: code 2 p (p < 4) or 2 (p - 4) + 1 of the word
    nib = nib.view(-1, K // 128, 4, 4, 2, 4).permute(0, 1, 3, 2, 5, 4)  # row, block, j, t, m, half
    w = (nib.reshape(-1, K).to(F32) - 8.0).view(-1, K // group, group) * sf.to(F32).reshape(-1, K // group, 1)
    return w.view(*q.shape[:-1], K)


def _plain_matvec(s):
    return (s["x"].to(F32) @ _plain_weights(s["q"], s["sf"], s["case"]["group"]).t()).to(BF16)


def _plain_experts(s):
    case = s["case"]
    T, H, I, k, group = (case[n] for n in ("T", "H", "I", "k", "group"))
    e = s["topk_idx"].reshape(-1).long()
    x = s["x"].to(F32).repeat_interleave(k, dim=0).unsqueeze(2)  # one row per slot
    h = torch.bmm(_plain_weights(s["W1_q"][e], s["W1_sf"][e], group), x).squeeze(2)
    a = h[:, :I] / (1.0 + torch.exp(-h[:, :I])) * h[:, I:]
    o = torch.bmm(_plain_weights(s["W2_q"][e], s["W2_sf"][e], group), a.unsqueeze(2)).view(T, k, H)
    return (o * s["topk_w"].unsqueeze(2)).sum(dim=1).to(BF16)


# ------------------------------------------------------- floors and 64 bits
def work(case):
    op = case["op"]
    if op == "norm":
        n, es = case["rows"] * case["H"], 4 if case["type"] == "f32" else 2
        step = case["dir"] == "step"
        return {"bytes": n * es * (4 if step else 2) + 8 * case["H"] * (2 if step else 1), "flops": n * (20 if step else 8)}
    if op == "ffn":
        T, H, I = case["T"], case["H"], case["I"]
        step = case["dir"] == "step"
        return {"bytes": 2 * (3 * H * I + 2 * T * H) + (2 * (3 * H * I + 2 * T * H) if step else 0),
                "flops": (18 if step else 6) * T * H * I}
    if op == "matvec":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": N * K / 2 + 2 * N * K / case["group"] + 2 * T * (N + K), "flops": 2 * T * N * K}
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    used = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token picks, each read once
    return {"bytes": used * 3 * H * I * (0.5 + 2 / case["group"]) + 4 * T * H + 8 * T * k, "flops": 6 * T * k * H * I}


def _weights64(q, sf, group):
    """float64 [N, K] of one matrix, code by code as the format states."""
    N, K = q.shape[0], 2 * q.shape[1]
    kk = torch.arange(K, device=q.device)
    b, r = kk // 128, kk % 128
    j, t, i = r // 32, (r % 32) // 8, r % 8
    nibble = 8 * (16 * b + 4 * t + j) + i // 2 + 4 * (i % 2)
    byte = q[:, nibble // 2].to(torch.int16)
    code = torch.where((nibble % 2 == 1)[None, :], byte >> 4, byte & 15)
    return (code - 8).double() * sf.double().repeat_interleave(group, dim=1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "norm":
        out = {}
        x, w = s["x"].double(), s["weight"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        inv = 1.0 / torch.sqrt(var + s["eps"])
        z = (x - mean) * inv
        out["y"] = z * w + (0.0 if s["bias"] is None else s["bias"].double())
        if case["dir"] == "step":
            dy = s["dy"].double()
            u = dy * w
            n = case["H"]
            out["dx"] = (u - (u.sum(1, True) + z * torch.einsum("rh,rh->r", u, z)[:, None]) / n) * inv
            out["dweight"] = torch.einsum("rh,rh->h", dy, z)
            if s["bias"] is not None:
                out["dbias"] = torch.einsum("rh->h", dy)
        return out
    if op == "ffn":
        I = case["I"]
        x, W1, W2 = s["x"].double(), s["W1"].double(), s["W2"].double()
        g, u = torch.mm(x, W1[:, :I]), torch.mm(x, W1[:, I:])
        sg = torch.sigmoid(g)
        a = g * sg * u
        out = {"y": torch.mm(a, W2)}
        if case["dir"] == "step":
            dy = s["dy"].double()
            da = torch.einsum("th,ih->ti", dy, W2)
            dg, du = da * u * (sg + g * sg * (1 - sg)), da * g * sg
            out["dW2"] = torch.einsum("ti,th->ih", a, dy)
            out["dx"] = torch.einsum("ti,hi->th", dg, W1[:, :I]) + torch.einsum("ti,hi->th", du, W1[:, I:])
            out["dW1"] = torch.cat((torch.einsum("th,ti->hi", x, dg), torch.einsum("th,ti->hi", x, du)), dim=1)
        return out
    if op == "matvec":
        return torch.einsum("tk,nk->tn", s["x"].double(), _weights64(s["q"], s["sf"], case["group"]))
    I, group = case["I"], case["group"]
    y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
    for e in torch.unique(s["topk_idx"]).tolist():
        t, slot = torch.nonzero(s["topk_idx"] == e, as_tuple=True)
        h = s["x"][t].double() @ _weights64(s["W1_q"][e], s["W1_sf"][e], group).t()
        a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
        o = a @ _weights64(s["W2_q"][e], s["W2_sf"][e], group).t()
        y.index_add_(0, t, o * s["topk_w"][t, slot].double()[:, None])
    return y
