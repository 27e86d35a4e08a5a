"""The joint's FP32 backward with many rows, whose groups have to be fewer than the
threads allow (test_residual_norm_plan_cpu has the plan): against 64 bits, rows on
16-byte boundaries and off them, and replayed to the bit."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from test_gpu_residual_norm import F32, _case, _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


@pytest.mark.parametrize("rows,H,options", [
    (3497, 128, dict()), (5000, 250, dict(kind="rms", gate="token")), (4001, 33, dict(gate="token")), (1825, 512, dict(gate="none")),
    (1300, 760, dict(post=False, gate="token")), (1000, 1024, dict(kind="rms", bias=False, post_bias=False, gate="none")),
    (1000, 1021, dict()), (470, 1700, dict(gate="token")), (460, 1537, dict(kind="rms", post=False, gate="none", bias=False)),
    (160, 3584, dict()), (153, 3500, dict(kind="rms", gate="token")), (300, 3333, dict(gate="token"))])
def test_many_rows(rows, H, options):
    c, ds, dn = _case(rows, H, F32, **options)
    first = _check(c, ds, dn)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _run(c, ds, dn)
    for v in out.values():
        v.fill_(5.0)
    g.replay()
    assert all(torch.equal(first[n], out[n]) for n in first)


@pytest.mark.parametrize("rows,H", [(184, 128), (185, 128), (368, 128), (369, 128), (48, 1024), (49, 1024), (96, 1024), (97, 1024)])
def test_around_the_cluster_of_few_rows(rows, H):
    _check(*_case(rows, H, F32, gate="token"))
