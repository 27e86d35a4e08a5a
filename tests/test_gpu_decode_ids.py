"""A given routing's expert ids, of every integer type: the int32 ids' outputs, to the bit."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.layer import DecodeLayer
from test_gpu_decode import _check_layer, _weights, _x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int8, torch.int16, torch.int64])
@pytest.mark.parametrize("E", [8, 128, 200])
def test_the_same_outputs_for_ids_of_any_type(dtype, E):
    T, k = 6, 3
    _, W1, W2, S1, S2 = _weights(64, 64, E, 64)
    x, g = _x(T, 64), torch.Generator(device="cuda").manual_seed(E)
    idx = torch.randint(0, min(E + 2, torch.iinfo(dtype).max + 1), (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randn(T, k, generator=g, device="cuda")
    for s1, s2 in ((None, None), (S1, S2)):
        layer = DecodeLayer(None, W1, W2, k, s1, s2)
        want = layer(x, idx, w)
        _check_layer(want, x, idx, w, W1, W2, s1, s2)
        assert want.any() and torch.equal(layer(x, idx.to(dtype), w), want)


def test_ids_of_other_types_are_refused():
    _, W1, W2, _, _ = _weights(64, 64, 8)
    layer, x, w = DecodeLayer(None, W1, W2, 2), _x(3, 64), torch.rand(3, 2, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        with pytest.raises(TypeError):
            layer(x, torch.zeros(3, 2, device="cuda", dtype=dtype), w)
