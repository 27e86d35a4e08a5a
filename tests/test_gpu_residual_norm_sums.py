"""Rows of more than 2048 columns: the sums of more than eight warps, one, two and
three of them in turn (test_residual_norm_sums_cpu has their places in shared memory).
Against 64 bits, and the same to the bit however often it is called."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from test_gpu_residual_norm import BF, F16, F32, _case, _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


@pytest.mark.parametrize("rows,H,options", [
    (1000, 2056, dict()), (1000, 4096, dict(gate="token")), (500, 7168, dict(wt=BF)), (500, 7168, dict(kind="rms", gate="token")),
    (900, 3000, dict(t=F16, gate="token", post=False, bias=False)), (300, 2400, dict(t=F32, gate="none")),
    (900, 4096, dict(post=False, gate="token")), (300, 2051, dict(gate="token"))])
def test_sums_of_changing_number(rows, H, options):
    c, ds, dn = _case(rows, H, **options)
    first = _check(c, ds, dn)
    for _ in range(30):
        again = _run(c, ds, dn)
        assert all(torch.equal(first[n], again[n]) for n in first)
