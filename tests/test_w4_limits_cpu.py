"""4-bit products: sizes past the kernels' 32-bit indexes are refused, and none
is cut to its low bits."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import W4Experts, W4Linear, quantize_w4

P = [4096 * (i + 1) for i in range(8)]  # addresses that no call may read


@pytest.mark.parametrize("N", [(1 << 30) + 1, (1 << 31) - 1])
def test_output_width(N):
    build.build()
    assert B.lib().moe_matvec_w4(1, N, 128, 32, *P[:4], None) == B.MOE_EUNSUPPORTED
    assert B.lib().moe_quantize_w4(1, 128, N, 32, *P[:3], None) == B.MOE_EUNSUPPORTED


class Sized:
    """What the constructors ask of a CUDA tensor."""

    is_cuda = True

    def __init__(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype

    def get_device(self):
        return 0

    def contiguous(self):
        return self


@pytest.mark.parametrize("N,K", [(1, (1 << 32) + 128), (1, 65536 + 128), ((1 << 32) + 8, 128), ((1 << 30) + 1, 128)])
def test_weights_past_the_limits(N, K):
    with pytest.raises(B.MoeError):
        W4Linear(Sized((N, K // 2), torch.uint8), Sized((N, K // 64), torch.bfloat16), 64)
    with pytest.raises(B.MoeError):
        quantize_w4(torch.empty((1, 1), dtype=torch.bfloat16).expand(K, N), 64)
    with pytest.raises(B.MoeError):
        B.moe_matvec_w4(Sized((1, K), torch.bfloat16), Sized((N, K // 2), torch.uint8), None, None, 64)
    if K > 65536:
        with pytest.raises(B.MoeError):
            W4Experts(Sized((1, 256, K // 2), torch.uint8), Sized((1, 256, K // 64), torch.bfloat16),
                      Sized((1, K, 64), torch.uint8), Sized((1, K, 2), torch.bfloat16), 64)


def test_weights_at_the_limits():
    W4Linear(Sized((1 << 30, 64), torch.uint8), Sized((1 << 30, 2), torch.bfloat16), 64)
    W4Linear(Sized((1, 32768), torch.uint8), Sized((1, 1024), torch.bfloat16), 64)
