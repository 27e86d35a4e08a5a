"""Up to 16 tokens the decoding layer's activations go into the down projection as two
bf16 numbers, the second the rest of the first's rounding: 16 significant bits.

First parts that cancel.  Two features, W2 of +1 and -1, activations a silu(16) with
a = 1 + 2^-9 and 1 - 2^-10: in bf16 (steps of 2^-7 above 1, 2^-8 below) both are 1, so
y is the rests alone, 16 (2^-9 + 2^-10).  silu(16) is 16 (1 - 1.2e-7).  The gate and up
projections are exact here (one and two products of powers of two).  A rest is at most 2^-8 of
its activation and is rounded to bf16 (2^-8 of itself: 2^-16 of 16 each), the
activation errs by 2^-18 of itself (device exp and divide, as in test_gpu_decode), which
its rest takes over; y is rounded by 2^-8 of itself.  A layer without the second part gives 0.

Any layer of up to 16 tokens.  As in test_gpu_decode, with 2^-16 for the activation's rounding
in the place of bf16's half step."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.layer import DecodeLayer
from test_gpu_decode import A, BF, HALF, _weights, _x

pytestmark = pytest.mark.gpu
REST = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


@pytest.mark.parametrize("T", [1, 8, 9, 16])
@pytest.mark.parametrize("shared", [False, True])
def test_first_parts_that_cancel(T, shared):
    H, I = 64, 72
    f = (5, 70)  # features of two tiles
    x = torch.zeros(T, H, device="cuda", dtype=BF)
    x[:, :2] = 1.0
    W1, W2 = torch.zeros(1, H, 2 * I, device="cuda", dtype=BF), torch.zeros(1, I, H, device="cuda", dtype=BF)
    W1[0, 0, f[0]], W1[0, 0, f[1]] = 16.0, 16.0
    W1[0, 0, I + f[0]], W1[0, 1, I + f[0]] = 1.0, 2.0 ** -9
    W1[0, 0, I + f[1]], W1[0, 1, I + f[1]] = 1.0, -(2.0 ** -10)
    W2[0, f[0]], W2[0, f[1]] = 1.0, -1.0
    idx, w = torch.zeros(T, 1, device="cuda", dtype=torch.int32), torch.ones(T, 1, device="cuda")
    if shared:  # the routed expert dropped
        y = DecodeLayer(None, W1, W2, 1, W1[0], W2[0])(x, idx - 1, w)
    else:
        y = DecodeLayer(None, W1, W2, 1)(x, idx, w)
    want = 16 * (2.0 ** -9 + 2.0 ** -10)
    assert ((y.double() - want).abs() <= 2 * 16 * (REST + 2.0 ** -18) + HALF * want).all()


def _expert(x, W1, W2):
    x, W1, W2 = x.double(), W1.double(), W2.double()
    h, eh = x @ W1, A * (x.abs() @ W1.abs())
    g, u = h.chunk(2, 1)
    eg, eu = eh.chunk(2, 1)
    s = g * torch.sigmoid(g)
    a = s * u
    return a @ W2, (1.1 * eg * u.abs() + s.abs() * eu + (REST + 2.0 ** -18 + A) * a.abs()) @ W2.abs()


@pytest.mark.parametrize("T,H,I,E,k,Is", [(1, 256, 128, 8, 2, 0), (8, 264, 136, 5, 3, 72), (16, 1024, 512, 16, 2, 512), (13, 520, 72, 33, 5, 0)])
def test_layers_of_up_to_16_tokens(T, H, I, E, k, Is):
    router, W1, W2, S1, S2 = _weights(H, I, E, Is, T)
    x = _x(T, H)
    y, idx, w = DecodeLayer(router, W1, W2, k, S1, S2)(x, return_routing=True)
    parts = []
    for t in range(T):
        for j in range(k):
            e, ww = int(idx[t, j]), float(w[t, j])
            parts.append((t, *(ww * v for v in _expert(x[t:t + 1], W1[e], W2[e]))))
        if Is:
            parts.append((t, *_expert(x[t:t + 1], S1, S2)))
    want, tol, size = (torch.zeros(T, H, dtype=torch.float64, device="cuda") for _ in range(3))
    for t, v, ev in parts:
        want[t] += v[0]
        tol[t] += ev[0]
        size[t] += v[0].abs()
    err = (y.double() - want).abs()
    assert (err <= tol + 2.0 ** -20 * size + HALF * (want.abs() + tol) + 1e-30).all()
