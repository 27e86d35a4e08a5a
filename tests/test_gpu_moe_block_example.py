"""The example block: norm, router, routed experts and the dense gated block
trained together and decoded with 4-bit experts."""
import importlib.util
import os

import pytest
import torch

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


def test_block_trains_and_decodes(example):
    block = example.MoEBlock(256, 128, 8, 2)
    x, losses = example.train(block, 300, 20)
    assert all(torch.isfinite(torch.tensor(losses))) and losses[-1] < 0.9 * losses[0]
    decode = example.W4Block(block, group=32)
    with torch.no_grad():
        want = block(x)
        one = torch.cat([decode(x[t: t + 1]) for t in range(6)])
        many = decode(x[:6])
    # one token at a time and together: the same sums, a few roundings apart in the router's products
    assert float((one.float() - many.float()).norm()) <= 0.02 * float(many.float().norm())
    # 4-bit weights err by at most half a step of max|w| / 7: about 0.1 of a normal weight's size, rms
    update = (want[:6] - x[:6]).float()
    assert float((many.float() - want[:6].float()).norm()) <= 0.35 * float(update.norm())


def test_gradients_of_the_whole_block(example):
    """d loss / d t along a direction, by central differences of the bf16 block's own loss.

    Only the FP32 parameters (norm weight and bias) can move by a small step exactly; the loss errs by bf16 roundings
    of about 2^-9 of its terms, independent over 300 x 128 of them, so a quotient over a step of 0.05 |p| is good to a
    few percent of its size."""
    block = example.MoEBlock(128, 64, 4, 2, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(300, 128, generator=g, device="cuda").to(torch.bfloat16)
    c = torch.randn(300, 128, generator=g, device="cuda")

    def loss():
        n = example.layer_norm(x, block.norm_w, block.norm_b)
        ws = block.workspaces(300)
        idx, w = fixed
        return ((example.moe_layer(n, block.W1, block.W2, idx, w, workspace=ws[0])
                 + example.gated_ffn(n, block.S1, block.S2, ws[1])).float() * c).sum()

    with torch.no_grad():
        fixed = block.route(example.layer_norm(x, block.norm_w, block.norm_b))
    loss().backward()
    for p in (block.norm_w, block.norm_b):
        d = p.grad / p.grad.norm()
        e = 0.3
        with torch.no_grad():
            p += e * d
            up = loss()
            p -= 2 * e * d
            down = loss()
            p += e * d
        got, want = float(p.grad.norm()), float((up - down) / (2 * e))
        assert abs(got - want) <= 0.1 * abs(want)
