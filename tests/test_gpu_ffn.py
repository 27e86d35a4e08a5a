"""The dense gated feed-forward block against 64 bits.

Tolerances, element by element, from the roundings: an FP32 accumulation of K
products in groups of 16 errs by at most about sqrt(K) / 16 * 2^-22 of the sum
of the products' sizes for the K used here: A = 2^-19 |x||w|.  a, dh and the
outputs are rounded to bf16 once (unit roundoff 2^-8: 8-bit significands).
The device exp errs by 2^-20 relative: 2^-18 |a| covers it.  |silu'| <= 1.1,
|silu''| <= 0.5.  These bounds add up worst cases; so each output's error in
the 2-norm is bounded too: three independent roundings at most, each at
most 2^-8 / sqrt(3) = 2.3e-3 rms of a value at the foot of its binade and 1.6e-3
over a whole binade, are below 3e-3 of the output's norm.  That is an average
over independent roundings: it holds where a row has at least 64 of them (at H =
I = 8 and one token the norm of dW1 is one or two values', whose two roundings
may err by 7.8e-3)."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import FFNWorkspace, ffn_backward, ffn_forward, gated_ffn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
A = 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


def _inputs(T, H, I, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)

    return n((T, H), 1.0), n((H, 2 * I), H ** -0.5), n((I, H), I ** -0.5), n((T, H), 1.0)


def _ref(x, W1, W2, dy, c=0.0):
    """{name: (value, tolerance)} in 64 bits."""
    x, W1, W2, dy = (t.double() for t in (x, W1, W2, dy))
    I = W2.shape[0]
    h, eh = x @ W1, A * (x.abs() @ W1.abs())
    g, u, eg, eu = h[:, :I], h[:, I:], eh[:, :I], eh[:, I:]
    pg, pu = torch.ones_like(g), torch.ones_like(u)
    if c > 0:
        pg, pu = (g.abs() <= c).double(), (u.abs() <= c).double()
        g, u = g.clamp(-c, c), u.clamp(-c, c)
    s = torch.sigmoid(g)
    ds = s * (1 + g * (1 - s))
    a = g * s * u
    ea = 1.1 * eg * u.abs() + (g * s).abs() * eu + (2.0 ** -8 + 2.0 ** -18) * a.abs()
    da, eda = dy @ W2.t(), A * (dy.abs() @ W2.abs().t())
    dh = torch.cat((pg * da * u * ds, pu * da * g * s), 1)
    edg = eda * (u * ds).abs() + da.abs() * (eu * ds.abs() + 0.5 * eg * u.abs() + 2.0 ** -19 * u.abs() * (1 + g.abs()))
    edu = eda * (g * s).abs() + da.abs() * (1.1 * eg + 2.0 ** -19 * (1 + g.abs()))
    edh = torch.cat((pg * edg, pu * edu), 1) + 2.0 ** -8 * dh.abs()

    def out(p, ep, q):
        v = p @ q
        return v, ep @ q.abs() + A * (p.abs() @ q.abs()) + 2.0 ** -8 * v.abs()

    r = dict(y=out(a, ea, W2), dx=out(dh, edh, W1.t()))
    for n, (l, p, ep) in dict(dW2=(dy, a, ea), dW1=(x, dh, edh)).items():
        v, e = out(p.t(), ep.t(), l)
        r[n] = (v, e) if n == "dW2" else (v.t(), e.t())
    near = torch.zeros_like(g, dtype=torch.bool) if c <= 0 else ((h.abs() - c).abs() <= 4 * eh)
    return r, near


def _close(name, got, ref, many=True):
    want, tol = ref
    err = (got.double() - want).abs()
    assert got.shape == want.shape
    assert (err <= tol + 1e-30).all(), f"{name}: {float((err / (tol + 1e-30)).max())} of its bound"
    if min(want.shape) > 0 and many:
        assert float(err.norm()) <= 3e-3 * float(want.norm()), f"{name}: {float(err.norm() / want.norm())} of its norm"


def _run(x, W1, W2, dy, ws):
    y = ffn_forward(x, W1, W2, ws)
    dx, dW1, dW2 = ffn_backward(dy, x, W1, W2, ws)
    assert ws.status() == 0
    return dict(y=y, dx=dx, dW1=dW1, dW2=dW2)


@pytest.mark.parametrize("T,H,I", [
    (1, 8, 8), (1, 64, 64), (3, 72, 40), (8, 2048, 1408), (17, 520, 136), (128, 128, 64), (129, 136, 264),
    (256, 256, 128), (257, 512, 200), (777, 1160, 712), (1024, 640, 384), (513, 64, 2048), (40, 7168, 256),
    (2500, 328, 88), (2048, 2048, 1408),
])
def test_against_64_bits(T, H, I):
    x, W1, W2, dy = _inputs(T, H, I, T + H)
    got = _run(x, W1, W2, dy, FFNWorkspace(T, H, I))
    ref, _ = _ref(x, W1, W2, dy)
    for n, v in got.items():
        _close(n, v, ref[n], many=min(H, I) >= 64)


@pytest.mark.parametrize("T,H,I", [(5, 256, 128), (300, 256, 192)])
def test_clamp(T, H, I):
    """The clamp's decisions are compared where h is not within its own error of the bound."""
    c = 0.8
    x, W1, W2, dy = _inputs(T, H, I, 3)
    ws = FFNWorkspace(T, H, I, activation_clamp=c)
    y = ffn_forward(x, W1, W2, ws)
    dx, dW1, dW2 = ffn_backward(dy, x, W1, W2, ws)
    ref, near = _ref(x, W1, W2, dy, c)
    _close("y", y, ref["y"])
    _close("dW2", dW2, ref["dW2"])
    _close("dW1", dW1[:, ~near.any(0)], tuple(t[:, ~near.any(0)] for t in ref["dW1"]))
    _close("dx", dx[~near.any(1)], tuple(t[~near.any(1)] for t in ref["dx"]))


def test_inference_form_and_guards():
    """Without train nothing past a is written; nothing around the outputs either."""
    T, H, I = 70, 136, 72
    x, W1, W2, dy = _inputs(T, H, I, 4)
    ws = FFNWorkspace(T, H, I, train=False)
    y = ffn_forward(x, W1, W2, ws)
    full = FFNWorkspace(T, H, I)
    guard = torch.full((T + 40, H), 3.0, dtype=BF, device="cuda")
    B.moe_ffn_forward(full.shape, x, W1, W2, full.saved, full.ws, guard[:T])
    assert torch.equal(y, guard[:T]) and (guard[T:] == 3.0).all()
    outs = [torch.full((n + 4096,), 3.0, dtype=BF, device="cuda") for n in (T * H, H * 2 * I, I * H)]
    B.moe_ffn_backward(full.shape, dy, x, W1, W2, full.saved, full.ws, *(o[:-4096] for o in outs))
    torch.cuda.synchronize()
    for o in outs:
        assert (o[-4096:] == 3.0).all()
    with pytest.raises(ValueError):
        ffn_backward(dy, x, W1, W2, ws)


def test_no_tokens():
    x, W1, W2, dy = _inputs(0, 64, 32)
    ws = FFNWorkspace(0, 64, 32)
    y = ffn_forward(x, W1, W2, ws)
    dx, dW1, dW2 = ffn_backward(dy, x, W1, W2, ws)
    assert y.shape == dx.shape == (0, 64) and not dW1.any() and not dW2.any()


def test_non_finite_rows_stay_in_their_row():
    T, H, I = 300, 128, 96
    x, W1, W2, _ = _inputs(T, H, I, 5)
    ws = FFNWorkspace(T, H, I)
    good = ffn_forward(x, W1, W2, ws)
    x2 = x.clone()
    x2[7, 3], x2[290, 0] = float("nan"), float("inf")
    y = ffn_forward(x2, W1, W2, ws)
    keep = [t for t in range(T) if t not in (7, 290)]
    assert torch.equal(y[keep], good[keep]) and y[7].isnan().all() and not torch.isfinite(y[290]).any()


@pytest.mark.parametrize("T", [6, 400])
def test_autograd_against_differences(T):
    H, I = 96, 64
    x, W1, W2, dy = _inputs(T, H, I, 6)
    p = [t.clone().requires_grad_() for t in (x, W1, W2)]
    y = gated_ffn(p[0].view(2, T // 2, H), p[1], p[2])
    y.backward(dy.view(2, T // 2, H))
    base = [t.double() for t in (x, W1, W2)]

    def f(x, W1, W2):
        h = x @ W1
        g = h[:, :I]
        return ((g * torch.sigmoid(g) * h[:, I:]) @ W2 * dy.double()).sum()

    for i in range(3):
        d = torch.randn(base[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64).cuda()
        d *= base[i].norm() / d.norm()
        e = 1e-5
        want = (f(*[b + e * d if j == i else b for j, b in enumerate(base)])
                - f(*[b - e * d if j == i else b for j, b in enumerate(base)])) / (2 * e)
        got = (p[i].grad.double() * d).sum()
        # the gradient errs by 3e-3 of its norm, along a direction of norm |d|
        assert abs(float(got - want)) <= 3e-3 * float(p[i].grad.double().norm() * d.norm())


def test_deterministic_other_stream_and_graph():
    T, H, I = 333, 256, 128
    x, W1, W2, dy = _inputs(T, H, I, 7)
    ws = FFNWorkspace(T, H, I)
    want = _run(x, W1, W2, dy, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = {n: v for n, v in zip(("y", "dx", "dW1", "dW2"),
                                    (ffn_forward(x, W1, W2, ws), *ffn_backward(dy, x, W1, W2, ws)))}
    torch.cuda.current_stream().wait_stream(s)
    for n in want:
        assert torch.equal(got[n], want[n])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = ffn_forward(x, W1, W2, ws)
        grads = ffn_backward(dy, x, W1, W2, ws)
    x.copy_(_inputs(T, H, I, 8)[0])
    g.replay()
    got = [t.clone() for t in (y, *grads)]
    want = _run(x, W1, W2, dy, ws)
    for a, n in zip(got, ("y", "dx", "dW1", "dW2")):
        assert torch.equal(a, want[n])


def test_stale_workspace_raises():
    x, W1, W2, dy = _inputs(8, 64, 32, 9)
    ws = FFNWorkspace(8, 64, 32)
    xr = x.clone().requires_grad_()
    y1 = gated_ffn(xr, W1, W2, ws)
    gated_ffn(xr, W1, W2, ws)
    with pytest.raises(RuntimeError):
        y1.backward(dy)


def test_refusals():
    with pytest.raises(B.MoeError):
        FFNWorkspace(4, 60, 64)
    with pytest.raises(B.MoeError):
        FFNWorkspace(4, 64, 20)
    with pytest.raises(B.MoeError):
        FFNWorkspace(-1, 64, 64)
    with pytest.raises(B.MoeError):
        FFNWorkspace(4, 64, 64, activation_clamp=float("inf"))
    x, W1, W2, dy = _inputs(4, 64, 32)
    ws = FFNWorkspace(4, 64, 32)
    with pytest.raises(ValueError):
        ffn_forward(x[:3], W1, W2, ws)
    with pytest.raises(TypeError):
        ffn_forward(x.float(), W1, W2, ws)
    with pytest.raises(ValueError):
        ffn_forward(x, W1.t().contiguous().t(), W2, ws)
    with pytest.raises(TypeError):
        ffn_forward(x.cpu(), W1, W2, ws)
    with pytest.raises(ValueError):
        ffn_backward(dy[:2], x, W1, W2, ws)


@pytest.mark.parametrize("T,H,I", [
    (2, 1160, 712),    # K in four parts, the last one shorter
    (9, 1160, 712),    # two jobs of eight tokens
    (16, 520, 136),
    (7, 16, 4104),     # one unit of K; a tile of eight features
    (9, 520, 2056),    # sixteen tokens a job, ragged tiles
    (16, 4096, 1024), (13, 2048, 1408), (15, 1032, 4096),
    (17, 1160, 712),   # three jobs of eight tokens
    (33, 2048, 1408), (96, 2048, 1408), (128, 512, 256), (127, 264, 72),
    (129, 512, 256), (100, 2048, 1408),  # the large form
    (4, 4096, 10248), (16, 4096, 10248),  # more tiles than SMs, K in four parts
    (3, 10248, 4096),  # the same in the down projection's tiles, K whole
    (5, 10248, 8200),  # and K in four parts
])
def test_few_tokens_forward(T, H, I):
    x, W1, W2, dy = _inputs(T, H, I, T + I)
    ws = FFNWorkspace(T, H, I, train=False)
    y = ffn_forward(x, W1, W2, ws)
    assert ws.status() == 0
    x64 = x.double()
    h, eh = x64 @ W1.double(), A * (x64.abs() @ W1.double().abs())
    g, u, eg, eu = h[:, :I], h[:, I:], eh[:, :I], eh[:, I:]
    s = torch.sigmoid(g)
    a = g * s * u
    ea = 1.1 * eg * u.abs() + (g * s).abs() * eu + (2.0 ** -8 + 2.0 ** -18) * a.abs()
    v = a @ W2.double()
    w = W2.double().abs()
    _close("y", y, (v, ea @ w + A * (a.abs() @ w) + 2.0 ** -8 * v.abs()), many=min(H, I) >= 64)


@pytest.mark.parametrize("T,H,I", [(5, 136, 72), (12, 136, 72), (11, 1032, 1096)])
def test_few_tokens_rows_and_guards(T, H, I):
    """Each row is its own token's alone, and nothing is written around the outputs."""
    x, W1, W2, _ = _inputs(T, H, I, 12)
    ws = FFNWorkspace(T, H, I)
    out = torch.full((T + 40, H), 3.0, dtype=BF, device="cuda")
    B.moe_ffn_forward(ws.shape, x, W1, W2, ws.saved, ws.ws, out[:T])
    good = ffn_forward(x, W1, W2, ws)
    assert torch.equal(out[:T], good) and (out[T:] == 3.0).all()
    x2 = x.clone()
    x2[1, 3], x2[4, H - 1] = float("nan"), float("inf")
    y = ffn_forward(x2, W1, W2, ws)
    keep = [t for t in range(T) if t not in (1, 4)]
    assert torch.equal(y[keep], good[keep]) and y[1].isnan().all() and not torch.isfinite(y[4]).any()


def test_few_tokens_clamped_training():
    """The h that the form for few tokens leaves, read by the backward."""
    H, I, c = 2048, 1408, 0.7
    x, W1, W2, dy = _inputs(16, H, I, 13)
    ws = FFNWorkspace(16, H, I, activation_clamp=c)
    y = ffn_forward(x, W1, W2, ws)
    dx, dW1, dW2 = ffn_backward(dy, x, W1, W2, ws)
    ref, near = _ref(x, W1, W2, dy, c)
    _close("y", y, ref["y"])
    _close("dW2", dW2, ref["dW2"])
    _close("dW1", dW1[:, ~near.any(0)], tuple(t[:, ~near.any(0)] for t in ref["dW1"]))
    _close("dx", dx[~near.any(1)], tuple(t[~near.any(1)] for t in ref["dx"]))
