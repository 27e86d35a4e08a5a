"""gated_ffn applies its workspace's clamp, or the call's own, and leaves the
workspace's as it is."""
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


@pytest.mark.parametrize("T", [7, 300])
def test_workspace_clamp_and_call_clamp(T):
    H, I, c = 256, 192, 0.5
    g = torch.Generator(device="cuda").manual_seed(1)

    def n(shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)

    x, W1, W2, dy = n((T, H), 1.0), n((H, 2 * I), H ** -0.5), n((I, H), I ** -0.5), n((T, H), 1.0)

    def plain(clamp):
        ws = FFNWorkspace(T, H, I, activation_clamp=clamp)
        return (ffn_forward(x, W1, W2, ws), *ffn_backward(dy, x, W1, W2, ws))

    def auto(*a, **k):
        p = [t.clone().requires_grad_() for t in (x, W1, W2)]
        y = gated_ffn(*p, *a, **k)
        y.backward(dy)
        return (y.detach(), *(t.grad for t in p))

    def same(a, b):
        return all(torch.equal(p, q) for p, q in zip(a, b))

    clamped, free, other = plain(c), plain(0.0), plain(0.9)
    assert not torch.equal(clamped[0], free[0]) and not torch.equal(other[0], clamped[0])
    ws, ws0 = FFNWorkspace(T, H, I, activation_clamp=c), FFNWorkspace(T, H, I)
    assert same(auto(ws), clamped) and same(auto(ws0), free) and same(auto(), free)
    # a call's own clamp holds for that call alone
    assert same(auto(ws, 0.9), other) and same(auto(ws, activation_clamp=0.0), free)
    assert same(auto(ws0, c), clamped) and same(auto(activation_clamp=c), clamped)
    assert torch.equal(ffn_forward(x, W1, W2, ws), clamped[0]) and torch.equal(ffn_forward(x, W1, W2, ws0), free[0])
    with torch.no_grad():
        assert torch.equal(gated_ffn(x, W1, W2, ws), clamped[0]) and torch.equal(gated_ffn(x, W1, W2, ws, 0.9), other[0])


def test_two_pending_calls_with_clamps_of_their_own():
    """Each backward takes the clamp of its own forward."""
    T, H, I = 40, 128, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((T, H), generator=g, device="cuda").to(BF)
    W1 = (torch.randn((H, 2 * I), generator=g, device="cuda") * H ** -0.5).to(BF)
    W2 = (torch.randn((I, H), generator=g, device="cuda") * I ** -0.5).to(BF)
    want = []
    for c in (0.4, 0.0):
        xr = x.clone().requires_grad_()
        gated_ffn(xr, W1, W2, activation_clamp=c).float().sum().backward()
        want.append(xr.grad)
    a, b = x.clone().requires_grad_(), x.clone().requires_grad_()
    wa, wb = FFNWorkspace(T, H, I, activation_clamp=0.4), FFNWorkspace(T, H, I)
    ya, yb = gated_ffn(a, W1, W2, wa), gated_ffn(b, W1, W2, wb)
    (ya.float().sum() + yb.float().sum()).backward()
    assert torch.equal(a.grad, want[0]) and torch.equal(b.grad, want[1])
