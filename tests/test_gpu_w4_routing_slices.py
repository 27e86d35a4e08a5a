"""Decoding token by token from a batch's routing: every slice of it is taken,
wherever it starts."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import W4Experts
from test_gpu_w4 import BF, _routing, _weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [1, 2, 3, 6])
def test_one_token_slices(k):
    build.build()
    T, H, I, E, G = 9, 256, 128, 8, 64
    ex = W4Experts(*_weights(2 * I, H, G, 1, E), *_weights(H, I, G, 2, E), G)
    x = torch.randn(T, H, device="cuda").to(BF)
    idx, w = _routing(T, E, k, 3)
    for n in (1, 2):
        for t in range(T - n + 1):
            s = slice(t, t + n)
            assert torch.equal(ex(x[s], idx[s], w[s]), ex(x[s].clone(), idx[s].clone(), w[s].clone())), (t, n)
