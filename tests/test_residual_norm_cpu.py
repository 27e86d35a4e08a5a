"""Host-side sizes and refusals of the residual joint: nothing here touches a device."""
import ctypes

import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import block, build

P = [4096 * (i + 1) for i in range(20)]  # addresses that no call may read
SHAPE = dict(rows=4, H=64, x_type=0, w_type=2, kind=0, gate=1, residual_scale=1.0, eps=1e-5)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def _shape(**kw):
    return ctypes.byref(B.MoeResidualNormShape(*{**SHAPE, **kw}.values()))


def _fwd(lib, shape=None, o=P[0], os=64, r=P[1], rs=64, g=P[2], pw=P[3], pb=P[4], w=P[5], b=P[6], s=P[7], n=P[8], st=P[9]):
    return lib.moe_residual_norm_forward(_shape(**(shape or {})), o, os, r, rs, g, pw, pb, w, b, s, n, st, None)


def _bwd(lib, shape=None, ds=P[0], dss=64, dn=P[1], dns=64, o=P[2], os=64, r=P[3], rs=64, g=P[4], pw=P[5], pb=P[6], w=P[7],
         st=P[8], ws=P[9], do=P[10], dr=P[11], dw=P[12], db=P[13], dpw=P[14], dpb=P[15], dg=P[16]):
    return lib.moe_residual_norm_backward(_shape(**(shape or {})), ds, dss, dn, dns, o, os, r, rs, g, pw, pb, w, st, ws, do, dr,
                                          dw, db, dpw, dpb, dg, None)


def test_declared_and_exported(lib):
    new = {"moe_residual_norm_forward", "moe_residual_norm_workspace", "moe_residual_norm_backward"}
    assert new <= set(B.declared_functions())
    assert all(hasattr(lib, n) for n in new)


@pytest.mark.parametrize("kw,code", [(dict(rows=-1), B.MOE_EINVAL), (dict(rows=1 << 31), B.MOE_EINVAL), (dict(H=0), B.MOE_EINVAL),
                                     (dict(H=(1 << 24) + 1), B.MOE_EINVAL), (dict(x_type=3), B.MOE_EUNSUPPORTED),
                                     (dict(w_type=1), B.MOE_EUNSUPPORTED), (dict(kind=2), B.MOE_EUNSUPPORTED),
                                     (dict(gate=3), B.MOE_EUNSUPPORTED), (dict(gate=-1), B.MOE_EUNSUPPORTED),
                                     (dict(residual_scale=float("nan")), B.MOE_EINVAL), (dict(eps=-1.0), B.MOE_EINVAL)])
def test_shapes(lib, kw, code):
    n = ctypes.c_size_t()
    assert lib.moe_residual_norm_workspace(_shape(**kw), ctypes.byref(n)) == code
    assert _fwd(lib, kw) == _bwd(lib, kw) == code


def test_arguments(lib):
    assert lib.moe_residual_norm_workspace(None, None) == B.MOE_EINVAL
    for kw in (dict(o=None), dict(r=None), dict(g=None), dict(pw=None), dict(w=None), dict(s=None), dict(n=None), dict(st=None),
               dict(os=63), dict(rs=8), dict(s=P[1], rs=72)):
        assert _fwd(lib, **kw) == B.MOE_EINVAL, kw
    for kw in (dict(o=P[0] + 1), dict(g=P[2] + 2), dict(w=P[5] + 2), dict(n=P[8] + 1), dict(st=P[9] + 2)):
        assert _fwd(lib, **kw) == B.MOE_EUNSUPPORTED, kw
    for kw in (dict(o=None), dict(r=None), dict(g=None), dict(pw=None), dict(w=None), dict(st=None), dict(do=None),
               dict(ws=None, shape=dict(rows=4000)), dict(dr=None), dict(dss=63), dict(dns=1), dict(os=63), dict(shape=dict(gate=0))):
        assert _bwd(lib, **kw) == B.MOE_EINVAL, kw
    for kw in (dict(ds=P[0] + 1), dict(dg=P[16] + 2), dict(ws=P[9] + 4), dict(dw=P[12] + 2)):
        assert _bwd(lib, **kw) == B.MOE_EUNSUPPORTED, kw
    assert _fwd(lib, dict(rows=0), o=None, w=None, s=None) == 0
    assert _bwd(lib, dict(rows=0), dw=None, db=None, dpw=None, dpb=None, dg=None) == 0


def test_sizes():
    def n(rows, H):
        return B.moe_residual_norm_workspace(B.residual_norm_shape(rows, H, torch.bfloat16, torch.float32))

    assert n(0, 64) == 0
    for rows, H in ((1, 1), (5, 64), (8, 2048), (40, 1024)):
        assert n(rows, H) == 0  # sums in one cluster
    for rows, H in ((4000, 64), (200, 2048), (9, 7168), (10 ** 6, 7168), (3, 40000), (10 ** 6, 40000)):
        assert min(rows, 8) * 16 * H <= n(rows, H) <= 152 * 16 * H
    assert n(10 ** 6, 1 << 24) <= 16 * 16 << 24


def test_python_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(TypeError):
        block.residual_norm_forward(x, x, w)  # not on a GPU
    with pytest.raises(TypeError):
        block.residual_norm_forward(x.double(), x.double(), w)
    for bad in (lambda: block.residual_norm_forward(x, x[:3], w), lambda: block.residual_norm_forward(x, x, w[:7]),
                lambda: block.residual_norm_forward(x, x, w, post_bias=w), lambda: block.residual_norm_forward(x, x, w, kind="l2"),
                lambda: block.residual_norm_forward(x, x, w, gate=torch.zeros(4)), lambda: block.residual_norm(x, x[0], w),
                lambda: block.residual_norm_backward(x[:3], x, x, x, w, torch.zeros(4, 4))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(B.MoeError):
        B.residual_norm_shape(1, 1 << 33, torch.float32, torch.float32)
