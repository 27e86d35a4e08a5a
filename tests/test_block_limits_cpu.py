"""Sizes past the kernels' 32-bit indexes are refused on the host."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build

P = [4096 * (i + 1) for i in range(16)]  # addresses that no call may read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


@pytest.mark.parametrize("H", [(1 << 29) + 1, 1 << 30, (1 << 31) - 1])
def test_layer_norm_width(lib, H):
    big = 1 << 40
    assert lib.moe_layer_norm_forward(1, H, 0, 2, P[0], big, P[1], P[2], 1e-5, P[3], P[4], P[5], None) == B.MOE_EINVAL
    assert lib.moe_layer_norm_backward(1, H, 0, 2, P[0], big, P[1], big, *P[2:10], None) == B.MOE_EINVAL
    assert lib.moe_layer_norm_forward(0, H, 0, 2, *([P[0], big] + P[1:3]), 1e-5, *P[3:6], None) == B.MOE_EINVAL
    with pytest.raises(B.MoeError):
        B.moe_layer_norm_workspace(1, H)


def test_layer_norm_width_at_the_limit():
    assert B.moe_layer_norm_workspace(1, 1 << 29) >= (1 << 29) * 8


@pytest.mark.parametrize("H", [(1 << 32) + 64, 1 << 32, (1 << 35) + 8])
def test_widths_past_the_c_type_are_not_cut(H):
    """Their low 32 bits would be another width."""
    with pytest.raises(B.MoeError):
        B.moe_layer_norm_workspace(1, H)
    x = torch.empty((1, 1), dtype=torch.bfloat16).expand(1, H)
    for call in (lambda: B.moe_layer_norm_forward(x, x, None, 1e-5, x, x, x),
                 lambda: B.moe_layer_norm_backward(x, x, x, x, x, x, x, None, x)):
        with pytest.raises(B.MoeError):
            call()
