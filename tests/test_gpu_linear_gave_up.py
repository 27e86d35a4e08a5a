"""A linear layer whose kernels give up on a wait: NaN in what they were to compute, the
status word set, and nothing written beside the outputs.  moe_selftest_give_up raises
the flag that such a wait raises; every wait still ends (nothing hangs or faults)."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import LinearWorkspace, linear, linear_backward, linear_forward

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
# few rows (one block a tile, several); K ranges and their join; tiles with and without
# residual and z, odd ends; gradients together, with a K split of their own
CASES = [(3, 64, 72, "silu", True), (8, 2048, 256, "gelu", True), (12, 4096, 1024, None, False), (300, 2048, 256, "silu", True),
         (777, 520, 4104, "gelu", True), (777, 520, 4104, None, True), (500, 72, 8200, None, False), (500, 72, 8200, "silu", False),
         (4096, 64, 72, "silu", False)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


@pytest.fixture
def giving_up():
    def switch(on):
        torch.cuda.synchronize()
        B.moe_selftest_give_up(on)

    yield switch
    switch(False)


def _inputs(T, K, N, residual):
    g = torch.Generator(device="cuda").manual_seed(T + K)

    def n(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(BF)

    return n(T, K), n(K, N), n(N), n(T, N) if residual else None, n(T, N)


@pytest.mark.parametrize("T,K,N,act,residual", CASES)
def test_outputs_are_nan_and_the_status_is_set(giving_up, T, K, N, act, residual):
    x, W, b, r, dy = _inputs(T, K, N, residual)

    def run(ws):
        y, z = linear_forward(x, W, b, r, act, True, ws)
        return y, z, *linear_backward(dy, x, W, z0 if z0 is not None else z, b, act, workspace=ws)

    z0 = None
    ws = LinearWorkspace(T, K, N, act)
    want = run(ws)
    z0 = want[1]  # the backward's column sums are of a forward that ended well
    assert ws.status() == 0 and all(v is None or v.isfinite().all() for v in want)
    giving_up(True)
    y, z, dx, dW, db = run(ws)
    assert ws.status() == 1
    assert y.isnan().all() and dx.isnan().all() and dW.isnan().all() and (z is None or z.isnan().all())
    assert torch.equal(db, want[4])  # sums that wait for nothing
    assert linear(x, W, b, r, act).isnan().all()  # without a workspace
    giving_up(False)
    ws = LinearWorkspace(T, K, N, act)
    assert all(v is w or torch.equal(v, w) for v, w in zip(run(ws), want)) and ws.status() == 0


@pytest.mark.parametrize("T,K,N,act,residual", CASES)
def test_nothing_is_written_beside_the_outputs(giving_up, T, K, N, act, residual):
    x, W, b, r, dy = _inputs(T, K, N, residual)
    s = B.linear_shape(T, K, N, act)
    pad = 4096

    def buffer(n, t=BF):
        return torch.full((n + pad,), 7.0, device="cuda", dtype=t)

    sizes = [B.moe_linear_workspace(s, back) for back in (False, True)]
    ws = torch.full((max(sizes) + pad,), 77, device="cuda", dtype=torch.uint8)
    ws[:16].zero_()
    y, z, dx, dW = buffer(T * N), buffer(T * N, torch.float32) if act else None, buffer(T * K), buffer(K * N)
    giving_up(True)
    B.moe_linear_forward(s, x, W, b, r, z, ws, y)
    assert (ws[sizes[0]:] == 77).all()
    B.moe_linear_backward(s, dy, x, W, z, ws, dx, dW, None)
    torch.cuda.synchronize()
    for v, n in ((y, T * N), (z, T * N), (dx, T * K), (dW, K * N)):
        if v is not None:
            assert v[:n].isnan().all() and (v[n:] == 7.0).all()
    assert (ws[max(sizes):] == 77).all()
