"""The stated input range of the 4-bit products: with G the group's length, the
sums carry up to 143 sum |x| over it, so |x| <= 1.8e34 stays finite for every
group (143 * 128 * 1.8e34 = 3.29e38, below the largest FP32, 3.40e38)."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import W4Linear
from test_gpu_w4 import BF, _check_product, _weights

pytestmark = pytest.mark.gpu

TOP = 1.8e34


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 100, 384), (5, 96, 1024), (12, 9000, 1408)])
def test_largest_inputs(M, N, K, G):
    build.build()
    q, sf = _weights(N, K, G, 7)
    q[0], q[1], q[2] = 0x00, 0xFF, 0x88  # every code 0, 15 and 8
    x = torch.full((M, K), TOP, device="cuda").to(BF)
    while float(x[0, 0]) > TOP:
        x = torch.nextafter(x, torch.zeros_like(x))
    if M > 1:
        x[1] = -x[1]
    if M > 2:
        x[2, ::2] = -x[2, ::2]
        x[3, K // 2:] = -x[3, K // 2:]
    y = W4Linear(q, sf, G)(x)
    assert torch.isfinite(y).all()
    _check_product(x, q, sf, G, y)
