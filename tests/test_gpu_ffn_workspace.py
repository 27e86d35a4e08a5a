"""What the dense gated feed-forward block keeps and writes: a stale workspace
is seen by the plain pair too, calls without gradients take the inference form,
pending backwards hold what is saved alone, and nothing lands past the buffers."""
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

    return n((T, H), 1.0), n((H, 2 * I), H ** -0.5), n((I, H), I ** -0.5), n((T, H), 1.0)


def test_plain_backward_of_an_overwritten_workspace():
    x, W1, W2, dy = _inputs(12, 64, 32, 1)
    ws = FFNWorkspace(12, 64, 32)
    ffn_forward(x, W1, W2, ws)
    first = ws.generation
    want = ffn_backward(dy, x, W1, W2, ws, generation=first)
    for a, b in zip(want, ffn_backward(dy, x, W1, W2, ws)):
        assert torch.equal(a, b)
    ffn_forward(dy, W1, W2, ws)
    with pytest.raises(RuntimeError):
        ffn_backward(dy, x, W1, W2, ws, generation=first)
    ffn_backward(dy, dy, W1, W2, ws, generation=ws.generation)
