"""The decoding layer's router where a cluster's eight blocks share the width
unevenly: narrow layers, where most of them have no row of it and reach their
exchange at once, and layers of more than 8192, where a block takes its range in
several passes.  Choice and weights as in 64 bits (test_gpu_decode's bounds, which
count H / 512 terms a thread); the outputs are those of the same layer with the
routing given, to the bit."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.layer import DecodeLayer
from test_gpu_decode import _check_routing, _weights, _x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


@pytest.mark.parametrize("T,H,E,k", [
    (1, 8, 33, 3), (9, 8, 40, 4), (64, 8, 1024, 8), (1, 56, 8, 2), (5, 56, 100, 5), (8, 64, 31, 2), (17, 120, 64, 6),
    (1, 8200, 16, 3), (9, 12344, 40, 4), (3, 16384, 33, 5), (1, 65536, 8, 2), (10, 65536, 8, 2)])
def test_widths_that_the_blocks_share_unevenly(T, H, E, k):
    router, W1, W2, _, _ = _weights(H, 8, E, seed=H)
    x = _x(T, H)
    layer = DecodeLayer(router, W1, W2, k)
    y, idx, w = layer(x, return_routing=True)
    _check_routing(x, router, idx, w, k)
    assert torch.equal(y, DecodeLayer(None, W1, W2, k)(x, idx, w))
    for _ in range(50 if H < 1000 else 3):  # the exchange, again and again
        assert all(torch.equal(a, b) for a, b in zip(layer(x, return_routing=True), (y, idx, w)))
