"""Host-side sizes and refusals of the linear layer: nothing here touches a device."""
import ctypes

import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import block, build

P = [4096 * (i + 1) for i in range(16)]  # addresses that no call may read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def _fwd(lib, shape=(4, 64, 72, 1), x=P[0], xs=64, W=P[1], b=P[2], bt=0, r=P[3], rs=72, z=P[4], ws=P[5], y=P[6]):
    return lib.moe_linear_forward(ctypes.byref(B.MoeLinearShape(*shape)), x, xs, W, b, bt, r, rs, z, ws, y, None)


def _bwd(lib, shape=(4, 64, 72, 1), dy=P[0], ds=72, x=P[1], xs=64, W=P[2], z=P[3], ws=P[4], dx=P[5], dW=P[6], db=P[7], bt=0):
    return lib.moe_linear_backward(ctypes.byref(B.MoeLinearShape(*shape)), dy, ds, x, xs, W, z, ws, dx, dW, db, bt, None)


def test_declared_and_exported(lib):
    new = {"moe_linear_workspace", "moe_linear_forward", "moe_linear_backward"}
    assert new <= set(B.declared_functions())
    assert all(hasattr(lib, n) for n in new)


@pytest.mark.parametrize("shape,code", [((4, 60, 64, 0), B.MOE_EUNSUPPORTED), ((4, 64, 20, 0), B.MOE_EUNSUPPORTED),
                                        ((-1, 64, 64, 0), B.MOE_EINVAL), ((4, 0, 64, 0), B.MOE_EINVAL),
                                        ((4, 64, -8, 0), B.MOE_EINVAL), ((4, 64, 64, 4), B.MOE_EUNSUPPORTED),
                                        ((4, 64, 64, -1), B.MOE_EUNSUPPORTED), ((4, 1 << 21, 64, 0), B.MOE_EUNSUPPORTED)])
def test_shapes(lib, shape, code):
    n = ctypes.c_size_t()
    assert lib.moe_linear_workspace(ctypes.byref(B.MoeLinearShape(*shape)), 0, ctypes.byref(n)) == code
    assert _fwd(lib, shape) == _bwd(lib, shape) == code


def test_arguments(lib):
    assert lib.moe_linear_workspace(None, 0, None) == B.MOE_EINVAL
    for kw in ({"x": None}, {"W": None}, {"ws": None}, {"y": None}, {"xs": 56}, {"rs": 64}, {"r": P[6], "rs": 80}):
        assert _fwd(lib, **kw) == B.MOE_EINVAL, kw
    for kw in ({"x": P[0] + 8}, {"b": P[2] + 2}, {"r": P[3] + 8}, {"z": P[4] + 4}, {"y": P[6] + 2}, {"xs": 68}, {"rs": 76},
               {"bt": 1}, {"bt": 3}, {"xs": 1 << 36}):
        assert _fwd(lib, **kw) == B.MOE_EUNSUPPORTED, kw
    for kw in ({"dy": None}, {"x": None}, {"W": None}, {"z": None}, {"ws": None}, {"ds": 64}, {"xs": 8}):
        assert _bwd(lib, **kw) == B.MOE_EINVAL, kw
    for kw in ({"dy": P[0] + 8}, {"dx": P[5] + 2}, {"dW": P[6] + 8}, {"db": P[7] + 2}, {"bt": 1}, {"ds": 76}):
        assert _bwd(lib, **kw) == B.MOE_EUNSUPPORTED, kw
    assert _fwd(lib, (0, 64, 72, 1), x=None, W=None, ws=None, y=None) == 0
    assert _bwd(lib, dx=None, dW=None, db=None) == 0
    assert _bwd(lib, (0, 64, 72, 1), dW=None, db=None) == 0


def test_sizes():
    for T, K, N, act in ((0, 64, 64, None), (1, 7168, 2048, "silu"), (777, 1160, 712, "gelu"), (8192, 2048, 7168, None)):
        s = B.linear_shape(T, K, N, act)
        fwd, bwd = B.moe_linear_workspace(s, False), B.moe_linear_workspace(s, True)
        assert fwd % 256 == bwd % 256 == 0 and fwd >= 256 and bwd >= 256 + (T * N * 2 if act else 0)
    assert B.moe_linear_workspace(B.linear_shape(8192, 2048, 7168), False) == 256  # a status word alone


def test_python_refusals():
    with pytest.raises(ValueError):
        B.linear_shape(4, 64, 64, "tanh")
    with pytest.raises(B.MoeError):
        B.linear_shape(1 << 40, 64, 64)
    x, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, 72, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        block.linear_forward(x, W)  # not on a GPU
    for bad in (lambda: block.linear_forward(x, W.t()), lambda: block.linear_forward(x[0], W),
                lambda: block.linear_forward(x, W, torch.zeros(71)), lambda: block.linear_backward(x, x, W)):
        with pytest.raises(ValueError):
            bad()
