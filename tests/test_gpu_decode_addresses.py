"""Weights whose storage is freed and made again between calls, as sharded training does
(test_decode_addresses_cpu has the addresses that the library is given)."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.layer import DecodeLayer
from test_gpu_decode import _weights, _x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


def test_weights_that_come_and_go():
    router, W1, W2, S1, S2 = _weights(64, 64, 8, 64)
    layer, x = DecodeLayer(router, W1, W2, 2, S1, S2), _x(6, 64)
    y, rows = layer(x), layer(x[::2])
    for name, t in (("router", router), ("W1", W1), ("W2", W2), ("S1", S1), ("S2", S2)):
        kept, storage = t.clone(), t.untyped_storage()
        size = storage.nbytes()
        torch.cuda.synchronize()
        storage.resize_(0)
        for form in (lambda: layer(x), lambda: layer(x[::2]), lambda: layer(x, return_routing=True)):
            with pytest.raises(RuntimeError, match=name):
                form()
        other = torch.full((size // 2,), float("nan"), device="cuda", dtype=torch.bfloat16)  # where it was, perhaps
        storage.resize_(size)
        t.copy_(kept)
        assert torch.equal(layer(x), y) and torch.equal(layer(x[::2]), rows)
        del other
