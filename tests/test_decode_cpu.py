"""Host-side sizes and refusals of the decoding layer: nothing here touches a device."""
import ctypes

import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.layer import DecodeLayer

P = [4096 * (i + 1) for i in range(12)]  # addresses that no call may read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def _fwd(lib, shape=(4, 64, 64, 8, 2, 64, 0.0), x=P[0], r=P[1], W1=P[2], W2=P[3], S1=P[4], S2=P[5], idx=P[6], w=P[7], ws=P[8],
         y=P[9]):
    return lib.moe_decode_forward(ctypes.byref(B.MoeDecodeShape(*shape)), x, r, W1, W2, S1, S2, idx, w, ws, y, None)


def test_declared_and_exported(lib):
    assert {"moe_decode_workspace", "moe_decode_forward"} <= set(B.declared_functions())
    assert hasattr(lib, "moe_decode_workspace") and hasattr(lib, "moe_decode_forward")


@pytest.mark.parametrize("shape,code", [
    ((-1, 64, 64, 8, 2, 0, 0.0), B.MOE_EINVAL), ((4, 0, 64, 8, 2, 0, 0.0), B.MOE_EINVAL), ((4, 64, 64, 8, 2, -8, 0.0), B.MOE_EINVAL),
    ((4, 64, 64, 0, 1, 0, 0.0), B.MOE_EINVAL), ((4, 64, 64, 1025, 1, 0, 0.0), B.MOE_EINVAL), ((4, 64, 64, 8, 9, 0, 0.0), B.MOE_EINVAL),
    ((4, 64, 64, 8, 0, 0, 0.0), B.MOE_EINVAL), ((4, 64, 64, 8, 2, 0, float("nan")), B.MOE_EINVAL),
    ((4, 60, 64, 8, 2, 0, 0.0), B.MOE_EUNSUPPORTED), ((4, 64, 20, 8, 2, 0, 0.0), B.MOE_EUNSUPPORTED),
    ((4, 64, 64, 8, 2, 4, 0.0), B.MOE_EUNSUPPORTED), ((65, 64, 64, 8, 2, 0, 0.0), B.MOE_EUNSUPPORTED),
    ((64, 64, 64, 32, 17, 0, 0.0), B.MOE_EUNSUPPORTED), ((4, 1 << 17, 64, 8, 2, 0, 0.0), B.MOE_EUNSUPPORTED)])
def test_shapes(lib, shape, code):
    n = ctypes.c_size_t()
    assert lib.moe_decode_workspace(ctypes.byref(B.MoeDecodeShape(*shape)), ctypes.byref(n)) == code
    assert _fwd(lib, shape) == code


def test_arguments(lib):
    assert lib.moe_decode_workspace(None, None) == B.MOE_EINVAL
    for kw in (dict(x=None), dict(W1=None), dict(W2=None), dict(S1=None), dict(S2=None), dict(idx=None), dict(w=None), dict(ws=None),
               dict(y=None)):
        assert _fwd(lib, **kw) == B.MOE_EINVAL, kw
    for kw in (dict(x=P[0] + 8), dict(r=P[1] + 2), dict(W1=P[2] + 8), dict(S2=P[5] + 8), dict(idx=P[6] + 2), dict(w=P[7] + 1),
               dict(ws=P[8] + 8), dict(y=P[9] + 2)):
        assert _fwd(lib, **kw) == B.MOE_EUNSUPPORTED, kw
    assert _fwd(lib, (0, 64, 64, 8, 2, 0, 0.0), x=None, y=None) == 0


def test_sizes():
    assert B.moe_decode_workspace(B.MoeDecodeShape(0, 64, 64, 8, 2, 0, 0.0)) == 0
    for T, H, I, E, k, Is in ((1, 64, 64, 8, 2, 0), (1, 7168, 2048, 256, 8, 2048), (64, 2048, 1408, 64, 6, 2816), (64, 8, 8, 1024, 16, 0)):
        n = B.moe_decode_workspace(B.MoeDecodeShape(T, H, I, E, k, Is, 0.0))
        assert n % 256 == 0 and n >= T * k * (2 * I + 4 * H) + T * (4 * E + 2 * Is)


def test_python_refusals():
    W1, W2 = torch.zeros(8, 64, 128, dtype=torch.bfloat16), torch.zeros(8, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        DecodeLayer(None, W1, W2, 2)  # not on a GPU
    with pytest.raises(ValueError):
        DecodeLayer(None, W1, W2[:4], 2)
    with pytest.raises(ValueError):
        DecodeLayer(None, W1, W2, 2, S1=W1[0])
