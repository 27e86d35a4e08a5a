"""gated_ffn without gradients uses the caller's workspace whatever it was made
for, and without one keeps nothing for a backward."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import FFNWorkspace, ffn_backward, ffn_forward, gated_ffn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


def _inputs(T, H, I, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)

    return n((T, H), 1.0), n((H, 2 * I), H ** -0.5), n((I, H), I ** -0.5)


@pytest.mark.parametrize("T", [5, 700])
def test_workspace_without_train_is_used(T):
    H, I = 128, 64
    x, W1, W2 = _inputs(T, H, I, T)
    want = ffn_forward(x, W1, W2, FFNWorkspace(T, H, I))
    p = [t.clone().requires_grad_() for t in (x, W1, W2)]
    for train in (False, True):
        ws = FFNWorkspace(T, H, I, train=train)
        assert torch.equal(gated_ffn(x.view(1, T, H), W1, W2, ws)[0], want) and ws.generation == 1
        with torch.no_grad():
            y = gated_ffn(*p, ws)
        assert torch.equal(y, want) and not y.requires_grad and ws.generation == 2 and ws.status() == 0
    # a training workspace holds what the plain backward reads, after a call without gradients too
    dy = torch.ones_like(x)
    got = ffn_backward(dy, x, W1, W2, ws)
    ffn_forward(x, W1, W2, ws)
    assert all(torch.equal(a, b) for a, b in zip(got, ffn_backward(dy, x, W1, W2, ws)))
    # gradients need what such a workspace has no room for: they come all the same
    gated_ffn(*p, FFNWorkspace(T, H, I, train=False)).float().sum().backward()
    assert all(t.grad is not None for t in p)


def test_no_buffer_for_the_backward():
    T, H, I = 2048, 64, 2048
    x, W1, W2 = _inputs(T, H, I)
    L = B.moe_ffn_workspace_layout(B.MoeFFNShape(T, H, I, 0.0))
    gated_ffn(x, W1, W2)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    gated_ffn(x, W1, W2)
    torch.cuda.synchronize()
    used = torch.cuda.max_memory_allocated() - before
    # a, scratch and y; the caching allocator rounds each block up to at most 2 MB
    assert used <= L.h + L.ws_bytes + T * H * 2 + 3 * (2 << 20), (used, L.h, L.ws_bytes, L.saved_bytes)


def test_a_call_without_gradients_makes_a_pending_backward_raise():
    x, W1, W2 = _inputs(8, 64, 32)
    ws = FFNWorkspace(8, 64, 32)
    xr = x.clone().requires_grad_()
    y = gated_ffn(xr, W1, W2, ws)
    with torch.no_grad():
        gated_ffn(xr, W1, W2, ws)
    with pytest.raises(RuntimeError):
        y.float().sum().backward()
