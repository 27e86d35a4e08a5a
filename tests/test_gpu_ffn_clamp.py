"""The activation clamp of the dense gated feed-forward block: a NaN is not
clamped away, and the workspace's own clamp is the one that gated_ffn applies
unless the call gives another."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import FFNWorkspace, ffn_backward, ffn_forward

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


def _inputs(T, H, I, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)

    return n((T, H), 1.0), n((H, 2 * I), H ** -0.5), n((I, H), I ** -0.5), n((T, H), 1.0)


def _step(x, W1, W2, dy, c):
    ws = FFNWorkspace(*x.shape, W2.shape[0], activation_clamp=c)
    y = ffn_forward(x, W1, W2, ws)
    out = (y, *ffn_backward(dy, x, W1, W2, ws))
    assert ws.status() == 0
    return out


@pytest.mark.parametrize("T,H,I", [
    (6, 256, 128),       # few tokens, eight a job
    (16, 2048, 1408),    # sixteen a job; dh from partial sums
    (300, 256, 192),     # the large form
    (200, 4096, 512),    # gate and up, and dh, from partial sums
    (140, 1152, 3000),   # the down projection from partial sums
])
@pytest.mark.parametrize("c", [0.0, 0.8])
def test_nan_is_not_clamped(T, H, I, c):
    x, W1, W2, dy = _inputs(T, H, I, 21)
    y, dx, _, _ = _step(x, W1, W2, dy, c)
    x2 = x.clone()
    x2[T // 2, 3] = float("nan")
    y2, dx2, dW1, dW2 = _step(x2, W1, W2, dy, c)
    keep = [t for t in range(T) if t != T // 2]
    assert y2[T // 2].isnan().all() and dx2[T // 2].isnan().all()
    assert torch.equal(y2[keep], y[keep]) and torch.equal(dx2[keep], dx[keep])
    assert dW1.isnan().all() and dW2.isnan().all()
    W3 = W1.clone()
    W3[1, I + 3] = float("nan")  # one feature of the up projection, in every token
    y3, dx3, _, dW23 = _step(x, W3, W2, dy, c)
    assert y3.isnan().all() and dx3.isnan().all() and dW23[3].isnan().all()
