"""CPU-only checks of the entry points around the routed experts: host-side
sizes, and refusals before any device is touched."""
import ctypes

import pytest

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build

P = [4096 * (i + 1) for i in range(16)]  # addresses that no call may read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def test_declared_and_exported(lib):
    names = set(B.declared_functions())
    new = {"moe_layer_norm_forward", "moe_layer_norm_workspace", "moe_layer_norm_backward", "moe_ffn_workspace_layout",
           "moe_ffn_forward", "moe_ffn_backward", "moe_quantize_w4", "moe_matvec_w4", "moe_w4_workspace",
           "moe_forward_w4"}
    assert new <= names
    for n in new:
        assert hasattr(lib, n)


def test_sizes():
    assert B.moe_layer_norm_workspace(0, 64) == 0
    assert B.moe_layer_norm_workspace(5, 64) >= 5 * 2 * 64 * 4
    assert B.moe_layer_norm_workspace(10 ** 6, 7168) <= 304 * 2 * 7168 * 4
    L = B.moe_ffn_workspace_layout(B.MoeFFNShape(8192, 7168, 2048, 0.0))
    assert L.a == 0 and L.h >= 8192 * 2048 * 2 and L.saved_bytes >= L.h + 8192 * 4096 * 4
    assert L.dh >= 16 and L.part >= L.dh + 8192 * 4096 * 2 and L.ws_bytes >= L.part
    # few tokens: room for the partial sums of a K-split product
    few = B.moe_ffn_workspace_layout(B.MoeFFNShape(8, 7168, 2048, 0.0))
    assert few.ws_bytes - few.part >= 2 * 8 * 4096 * 4
    for T in (0, 1, 300):
        L = B.moe_ffn_workspace_layout(B.MoeFFNShape(T, 64, 40, 0.0))
        assert all(v % 256 == 0 for v in (L.h, L.dh, L.part, L.saved_bytes))
    assert B.moe_w4_workspace(B.MoeW4Shape(3, 256, 128, 8, 2, 32)) >= 6 * 128 * 2 + 6 * 256 * 4
    assert B.moe_w4_workspace(B.MoeW4Shape(0, 256, 128, 8, 2, 32)) == 0


def test_layer_norm_refusals(lib):
    f = lib.moe_layer_norm_forward

    def fwd(rows=4, H=64, xt=0, wt=2, x=P[0], xs=64, w=P[1], b=P[2], eps=1e-5, y=P[3], m=P[4], r=P[5]):
        return f(rows, H, xt, wt, x, xs, w, b, eps, y, m, r, None)

    assert fwd(rows=-1) == fwd(rows=1 << 31) == fwd(H=0) == fwd(xs=63) == B.MOE_EINVAL
    assert fwd(eps=float("nan")) == fwd(eps=-1.0) == fwd(x=None) == fwd(w=None) == fwd(m=None) == B.MOE_EINVAL
    assert fwd(xt=3) == fwd(wt=1) == fwd(xt=2, wt=0) == B.MOE_EUNSUPPORTED
    assert fwd(x=P[0] + 1) == fwd(m=P[4] + 2) == fwd(w=P[1] + 2) == B.MOE_EUNSUPPORTED
    assert fwd(rows=0, x=None, y=None) == 0
    g = lib.moe_layer_norm_backward

    def bwd(rows=4, xs=64, ds=64, dw=P[6], ws=P[8]):
        return g(rows, 64, 0, 2, P[0], ds, P[1], xs, P[2], P[3], P[4], P[5], dw, P[7], ws, None)

    assert bwd(xs=10) == bwd(ds=63) == bwd(dw=None) == bwd(ws=None) == B.MOE_EINVAL
    assert bwd(ws=P[8] + 4) == B.MOE_EUNSUPPORTED
    assert lib.moe_layer_norm_workspace(4, 64, None) == B.MOE_EINVAL


@pytest.mark.parametrize("shape,code", [((4, 60, 64, 0.0), B.MOE_EUNSUPPORTED), ((4, 64, 20, 0.0), B.MOE_EUNSUPPORTED),
                                        ((-1, 64, 64, 0.0), B.MOE_EINVAL), ((4, 0, 64, 0.0), B.MOE_EINVAL),
                                        ((4, 64, 64, float("nan")), B.MOE_EINVAL),
                                        ((4, 1 << 21, 64, 0.0), B.MOE_EUNSUPPORTED)])
def test_ffn_refusals(lib, shape, code):
    s, L = B.MoeFFNShape(*shape), B.MoeFFNLayout()
    assert lib.moe_ffn_workspace_layout(ctypes.byref(s), ctypes.byref(L)) == code
    assert lib.moe_ffn_forward(ctypes.byref(s), *P[:3], 1, *P[3:6], None) == code
    assert lib.moe_ffn_backward(ctypes.byref(s), *P[:9], None) == code


def test_ffn_pointers(lib):
    s = B.MoeFFNShape(4, 64, 64, 0.0)
    assert lib.moe_ffn_forward(ctypes.byref(s), None, *P[1:3], 1, *P[3:6], None) == B.MOE_EINVAL
    assert lib.moe_ffn_forward(ctypes.byref(s), P[0] + 8, *P[1:3], 1, *P[3:6], None) == B.MOE_EUNSUPPORTED
    assert lib.moe_ffn_backward(ctypes.byref(s), *P[:7], None, P[8], None) == B.MOE_EINVAL
    assert lib.moe_ffn_workspace_layout(None, None) == B.MOE_EINVAL
    z = B.MoeFFNShape(0, 64, 64, 0.0)
    assert lib.moe_ffn_forward(ctypes.byref(z), None, None, None, 1, None, None, None, None) == 0


def test_w4_refusals(lib):
    mv = lib.moe_matvec_w4
    assert mv(1, 8, 100, 32, *P[:4], None) == mv(1, 8, 128, 48, *P[:4], None) == B.MOE_EUNSUPPORTED
    assert mv(1, 8, 131072, 32, *P[:4], None) == mv(70000, 8, 128, 32, *P[:4], None) == B.MOE_EUNSUPPORTED
    assert mv(-1, 8, 128, 32, *P[:4], None) == mv(1, 0, 128, 32, *P[:4], None) == B.MOE_EINVAL
    assert mv(1, 8, 128, 32, None, *P[1:4], None) == B.MOE_EINVAL
    assert mv(1, 8, 128, 32, P[0] + 2, *P[1:4], None) == B.MOE_EUNSUPPORTED
    assert mv(0, 8, 128, 32, None, None, None, None, None) == 0

    def fwd(shape, idx=P[5], ws=P[7]):
        s = B.MoeW4Shape(*shape)
        return lib.moe_forward_w4(ctypes.byref(s), *P[:5], idx, P[6], ws, P[8], None)

    assert fwd((1, 100, 128, 8, 2, 32)) == fwd((1, 128, 64, 8, 2, 32)) == fwd((1, 128, 128, 8, 2, 16)) == B.MOE_EUNSUPPORTED
    assert fwd((9000, 128, 128, 8, 8, 32)) == B.MOE_EUNSUPPORTED
    assert fwd((1, 128, 128, 8, 9, 32)) == fwd((1, 128, 128, 8, 2, 32), idx=None) == B.MOE_EINVAL
    assert fwd((1, 128, 128, 8, 2, 32), ws=None) == fwd((-1, 128, 128, 8, 2, 32)) == B.MOE_EINVAL
    assert fwd((0, 128, 128, 8, 2, 32)) == 0
    assert lib.moe_w4_workspace(None, None) == B.MOE_EINVAL
    q = lib.moe_quantize_w4
    assert q(1, 100, 8, 32, *P[:3], None) == q(1, 128, 8, 100, *P[:3], None) == B.MOE_EUNSUPPORTED
    assert q(0, 128, 8, 32, *P[:3], None) == q(1, 128, 8, 32, None, *P[1:3], None) == B.MOE_EINVAL
