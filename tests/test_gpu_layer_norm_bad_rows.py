"""NaN and infinity in rows of the layer norm's persistent forms: groups of one
warp, with a reducing warp and with every warp reducing, each with rows on and
between vector boundaries.  Several rows pass through a group; what is not
finite stays in its row, and in the columns whose sums it belongs to."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import layer_norm_backward, layer_norm_forward

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("rows,H,t", [
    (7400, 128, BF), (7400, 512, F16), (7400, 1000, BF),  # one warp, 1, 2 and (forward) 4 vectors a thread
    (2400, 2048, BF), (1000, 7168, F16), (2400, 1024, F32),  # a reducing warp
    (1000, 8192, BF), (1000, 4096, F32),  # every warp reduces (backward)
    (8001, 33, BF), (8001, 251, F32),  # between vector boundaries: one warp
    (7400, 1001, F16), (2600, 2047, F32), (1400, 5003, BF),  # a reducing warp
    (1000, 8189, F16), (1000, 4101, F32),  # every warp
])
def test_what_is_not_finite_stays_where_it_belongs(rows, H, t):
    build.build()
    g = torch.Generator(device="cuda").manual_seed(rows + H)
    x = torch.randn((rows, H), generator=g, device="cuda").to(t)
    dy = torch.randn((rows, H), generator=g, device="cuda").to(t)
    w = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
    b = torch.randn(H, generator=g, device="cuda")
    y, mean, rstd = layer_norm_forward(x, w, b)
    dx, dw, db = layer_norm_backward(dy, x, w, mean, rstd)
    assert all(torch.isfinite(v).all() for v in (y, mean, rstd, dx, dw, db))
    # first and last rows, neighbours, rows of the same group; first and last columns and between
    at = {0: (0, NAN), 1: (H - 1, INF), 152: (H // 2, -INF), 304: (5, NAN), 760: (H - 2, NAN), rows - 1: (H - 1, NAN)}
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    x2 = x.clone()
    for r, (c, v) in at.items():
        x2[r, c], keep[r] = v, False
    y2, mean2, rstd2 = layer_norm_forward(x2, w, b)
    assert y2[~keep].isnan().all() and rstd2[~keep].isnan().all()
    for p, q in ((y, y2), (mean, mean2), (rstd, rstd2)):
        assert torch.equal(p[keep], q[keep])
    dx2, dw2, db2 = layer_norm_backward(dy, x2, w, mean2, rstd2)
    assert dx2[~keep].isnan().all() and torch.equal(dx2[keep], dx[keep])
    assert dw2.isnan().all() and torch.equal(db2, db)
    # in dy: the row's dx, and its own column's sums
    dy2 = dy.clone()
    cols = torch.ones(H, dtype=torch.bool, device="cuda")
    for r, (c, v) in at.items():
        dy2[r, c], cols[c] = v, False
    dx2, dw2, db2 = layer_norm_backward(dy2, x, w, mean, rstd)
    assert not torch.isfinite(dx2[~keep]).any() and torch.equal(dx2[keep], dx[keep])
    assert torch.equal(dw2[cols], dw[cols]) and torch.equal(db2[cols], db[cols])
    assert not torch.isfinite(dw2[~cols]).any() and not torch.isfinite(db2[~cols]).any()
