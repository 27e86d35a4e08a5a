"""Projections, joint, routed and shared experts run together, trained and decoded."""
import importlib.util
import os

import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _x(T, H, seed=4):
    return torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


def _reference(b, x, idx, w):
    """The block in 64 bits by autograd: (y, its parameters' copies)."""
    p = {n: getattr(b, n).detach().double().requires_grad_() for n in
         ("norm_w", "norm_b", "W1", "W2", "S1", "S2", "P1", "P2", "b1", "b2", "post_w", "gate")}

    def rms(v):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5)

    def expert(v, W1, W2):
        g, u = (v @ W1).chunk(2, 1)
        return (torch.nn.functional.silu(g) * u) @ W2

    x = x.double()
    m = torch.nn.functional.gelu(x @ p["P1"] + p["b1"]) @ p["P2"] + p["b2"]
    s = x + p["gate"] * (rms(m) * p["post_w"])
    n = rms(s) * p["norm_w"] + p["norm_b"]
    y = s + expert(n, p["S1"], p["S2"])
    for e in range(b.E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        y = y.index_add(0, t, expert(n[t], p["W1"][e], p["W2"][e]) * w[t, j].double()[:, None])
    return y, p


def test_gradients_of_the_block(example):
    """Every parameter's gradient against 64 bits, the routing's choice and weights held.

    A path through the block has at most 30 roundings to bf16, forward and backward, each at most 2^-8 / sqrt(3) = 2.3e-3
    of a tensor's norm (rms); independent, and through slopes of the order 1 (norms, activations), they add up to
    sqrt(30) 2.3e-3 = 1.3e-2, twice that with a slope of 2: the bound."""
    b = example.MixedBlock(256, 128, 8, 2, seed=3)
    x = _x(200, 256)
    with torch.no_grad():
        idx, w = b.route(b.first_half(x)[1])
    y = b(x, (idx, w))
    dy = _x(200, 256, 9)
    y.backward(dy)
    want, p = _reference(b, x, idx, w)
    want.backward(dy.double())
    assert float((y.double() - want).detach().norm()) <= 2.6e-2 * float(want.detach().norm())
    for n, v in p.items():
        got = getattr(b, n).grad
        assert got is not None and float((got.double() - v.grad).norm()) <= 2.6e-2 * float(v.grad.norm()), n


def test_trains_and_decodes(example):
    b = example.MixedBlock(128, 64, 8, 2)
    x, losses = example.train(b, 300, 3)
    assert all(torch.isfinite(torch.tensor(losses)))
    decode = b.decoder()
    with torch.no_grad():
        want, idx = b(x), b.route(b.first_half(x)[1])[0]
    one, many = torch.cat([decode(x[t: t + 1]) for t in range(12)]), decode(x[:12])
    # rows differ from form to form by their own roundings; a token whose k-th and next logit are as near as the example's
    # own bf16 router rounds them (2^-8 of their size) may take another expert in the two kernels' FP32 logits
    n = b.first_half(x[:12])[1]
    l = n.float() @ b.router.float()
    top = l.sort(1, descending=True).values
    clear = (top[:, 1] - top[:, 2]) > 2.0 ** -6 * (1 + top[:, 0].abs())
    assert int(clear.sum()) >= 6
    for got in (one, many):
        assert float((got[clear].float() - want[:12][clear].float()).norm()) <= 2.6e-2 * float(want[:12][clear].float().norm())
    assert idx.shape == (300, 2)


def test_decoding_captured_and_replayed(example):
    b = example.MixedBlock(128, 64, 8, 2, seed=5)
    decode, x = b.decoder(), _x(4, 128)
    want = decode(x)
    names = []
    with B.KernelTrace(16) as t:
        decode(x)
    torch.cuda.synchronize()
    names = t.names
    assert names == ["linear_few", "linear_few", "residual_norm_fwd", "decode_router", "decode_experts"]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = decode(x)
    for seed in (4, 8, 12):
        x.copy_(_x(4, 128, seed))
        g.replay()
        assert torch.equal(y, decode(x))
    assert torch.equal(want, decode(x.copy_(_x(4, 128))))
