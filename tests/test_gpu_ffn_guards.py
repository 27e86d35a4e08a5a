"""The forward without for_backward writes nothing past the activation in the
buffer of saved values, in every form of it."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("T,H,I", [
    (5, 136, 72),        # few tokens, eight a job
    (16, 2048, 1408),    # sixteen a job
    (70, 136, 72),       # several jobs
    (300, 256, 200),     # the large form
    (777, 1160, 712),
    (200, 4096, 520),    # gate and up from partial sums
    (140, 1152, 3000),   # the down projection from partial sums
])
def test_inference_leaves_the_rest_of_saved(T, H, I):
    build.build()
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((T, H), generator=g, device="cuda").to(BF)
    W1 = (torch.randn((H, 2 * I), generator=g, device="cuda") * H ** -0.5).to(BF)
    W2 = (torch.randn((I, H), generator=g, device="cuda") * I ** -0.5).to(BF)
    s = B.MoeFFNShape(T, H, I, 0.0)
    L = B.moe_ffn_workspace_layout(s)
    a_bytes = 2 * T * I
    saved = torch.full((L.saved_bytes + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = torch.full((L.ws_bytes + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    ws[:16] = 0
    y = torch.empty((T, H), dtype=BF, device="cuda")
    B.moe_ffn_forward(s, x, W1, W2, saved, ws, y, for_backward=False)
    torch.cuda.synchronize()
    assert (saved[a_bytes:] == 0x5A).all() and (ws[L.ws_bytes:] == 0x5A).all() and not ws[:16].any()
    full = torch.full((L.saved_bytes + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    y2 = torch.empty((T, H), dtype=BF, device="cuda")
    B.moe_ffn_forward(s, x, W1, W2, full, ws, y2, for_backward=True)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(saved[:a_bytes], full[:a_bytes])
    h = full[L.h: L.h + 8 * T * I].view(torch.float32).view(T, 2 * I)
    assert torch.isfinite(h).all() and (full[L.h + 8 * T * I:] == 0x5A).all() and (ws[L.ws_bytes:] == 0x5A).all()
