"""The experts with 4-bit weights under an activation clamp, against 64 bits.

Tolerance: test_gpu_w4's, with the clamped gate and up: a clamp moves an
argument's error through itself at most whole."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import W4Experts, quantize_w4
from test_gpu_w4 import BF, _decode, _routing, _weights

pytestmark = pytest.mark.gpu


def _ref(x, W1, W2, G, idx, w, c):
    T, H = x.shape
    y, tol = (torch.zeros(T, H, device="cuda", dtype=torch.float64) for _ in range(2))
    xd = x.double()
    clamped = 0
    for e in range(W1[0].shape[0]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if not len(t):
            continue
        c1, s1 = _decode(W1[0][e], W1[1][e], G)
        c2, s2 = _decode(W2[0][e], W2[1][e], G)
        I = c1.shape[0] // 2
        h, dh = xd[t] @ (c1 * s1).t(), 2.0 ** -20 * 280 * (xd[t].abs() @ s1.t())
        clamped += int((h.abs() > c).sum())
        g, u = h[:, :I].clamp(-c, c), h[:, I:].clamp(-c, c)
        sg = torch.sigmoid(g)
        a = g * sg * u
        da = 1.1 * dh[:, :I] * u.abs() + (g * sg).abs() * dh[:, I:] + (2.0 ** -8 + 2.0 ** -20) * a.abs()
        ww = w[t, j].double()[:, None]
        y.index_add_(0, t, ww * (a @ (c2 * s2).t()))
        tol.index_add_(0, t, ww.abs() * (da @ (c2 * s2).abs().t() + 2.0 ** -20 * 280 * (a.abs() @ s2.t())))
    assert clamped > 0
    return y, tol + 2.0 ** -8 * y.abs()


@pytest.mark.parametrize("T,H,I,E,k,G,c", [(1, 256, 128, 8, 2, 64, 0.7), (20, 512, 384, 4, 2, 32, 0.4),
                                           (9, 2048, 2816, 1, 1, 128, 1.0)])
def test_clamped_experts(T, H, I, E, k, G, c):
    build.build()
    W1, W2 = _weights(2 * I, H, G, 1, E), _weights(H, I, G, 2, E)
    x = torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(BF)
    idx, w = _routing(T, E, k, 5)
    ex = W4Experts(*W1, *W2, G, activation_clamp=c)
    y = ex(x, idx, w)
    want, tol = _ref(x, W1, W2, G, idx, w, c)
    err = (y.double() - want).abs()
    assert (err <= tol).all(), float((err / tol.clamp_min(1e-30)).max())
    if E == 1:  # a shared expert, without routing
        y = ex(x)
        want, tol = _ref(x, W1, W2, G, idx, torch.ones_like(w), c)
        assert ((y.double() - want).abs() <= tol).all()
    free = W4Experts(*W1, *W2, G)
    assert torch.equal(W4Experts(*W1, *W2, G, activation_clamp=1e30)(x, idx, w), free(x, idx, w))
    assert not torch.equal(free(x, idx, w), ex(x, idx, w))


def test_nan_is_not_clamped_and_refusals():
    build.build()
    H, I, G = 256, 128, 64
    g = torch.Generator(device="cuda").manual_seed(6)
    W1, W2 = (torch.randn(s, generator=g, device="cuda").to(BF) for s in ((H, 2 * I), (I, H)))
    ex = W4Experts.quantize(W1, W2, G, activation_clamp=0.5)
    x = torch.randn(3, H, generator=g, device="cuda").to(BF)
    good = ex(x)
    x[1, 7] = float("nan")
    y = ex(x)
    assert y[1].isnan().all() and torch.equal(y[[0, 2]], good[[0, 2]])
    for c in (float("nan"), float("inf")):
        with pytest.raises(B.MoeError):
            W4Experts(*quantize_w4(W1[None], G), *quantize_w4(W2[None], G), G, activation_clamp=c)(x)
