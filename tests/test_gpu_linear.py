"""The linear layer (bias, activation, residual) against 64 bits.

Tolerances, element by element, from the roundings.  z = x W + b: an FP32
accumulation of K products in groups of 16 errs by at most about sqrt(K) / 16 *
2^-22 of the sum of the products' sizes for the K used here, A = 2^-19 |x||W|,
and the bias's addition by 2^-24 (|z| + |b|) more: 2^-23 of both covers it.  The activations' slopes are
at most 1.13 and their second derivatives at most 0.8; their values err by
2^-18 (1 + |z|) of themselves (device exp and divide 2^-20, erfc 2^-20, the
argument's rounding times |z|), and by 2^-20 of their sizes with the residual's
addition.  y, dz, dx, dW and a bf16 db are rounded once each, half a step of
bf16: 2^-8 of the value.  db's sum of T terms in FP32 errs by at most (T + 64)
2^-24 of the sum of their sizes, whatever its order."""
import math

import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import LinearWorkspace, linear, linear_backward, linear_forward

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
A, HALF = 2.0 ** -19, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


def _act(z, act):
    """(act(z), act'(z)) in 64 bits."""
    if act is None:
        return z, torch.ones_like(z)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # (1 + tanh u) / 2 = sigmoid(2 u), which does not cancel where tanh nears -1
    c = math.sqrt(2 / math.pi)
    u = c * (z + 0.044715 * z ** 3)
    s, q = torch.sigmoid(2 * u), torch.sigmoid(2 * u) * torch.sigmoid(-2 * u)
    return z * s, s + 2 * z * q * c * (1 + 3 * 0.044715 * z * z)


def _inputs(T, K, N, seed=0, bias=BF, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(shape, std, t=BF):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(t)

    return (n((T, K), 1.0), n((K, N), K ** -0.5), None if bias is None else n((N,), 0.5, bias),
            n((T, N), 1.0) if residual else None, n((T, N), 1.0))


def _ref(x, W, b, r, dy, act):
    """{name: (value, tolerance)} in 64 bits."""
    db_t = None if b is None else b.dtype
    x, W, dy = x.double(), W.double(), dy.double()
    b = torch.zeros(W.shape[1], dtype=torch.float64, device="cuda") if b is None else b.double()
    p = x @ W
    z = p + b
    ez = A * (x.abs() @ W.abs()) + 2.0 ** -23 * (p.abs() + b.abs())
    a, s = _act(z, act)
    rel = 0.0 if act is None else 2.0 ** -18 * (1 + z.abs())
    ea = (1.0 if act is None else 1.13) * ez + rel * a.abs()
    y = a if r is None else a + r.double()
    ey = ea + 2.0 ** -20 * (a.abs() + (0 if r is None else r.double().abs())) + HALF * y.abs()
    dz = dy * s
    edz = dy.abs() * (0.0 if act is None else 0.8 * ez + rel * (s.abs() + 2.0 ** -6))
    out = {"y": (y, ey)}
    q = edz + (0.0 if act is None else HALF * dz.abs())  # as an operand
    for n, (l, el, m) in {"dx": (dz, q, W.t()), "dWt": (dz.t(), q.t() if torch.is_tensor(q) else q, x)}.items():
        v = l @ m
        out[n] = (v, el @ m.abs() + A * (l.abs() @ m.abs()) + HALF * v.abs())
    out["dW"] = tuple(t.t() for t in out.pop("dWt"))
    if db_t is not None:
        v = dz.sum(0)
        out["dbias"] = (v, edz.sum(0) + (len(dy) + 64) * 2.0 ** -24 * (dz.abs() + edz).sum(0)
                        + (HALF if db_t is BF else 2.0 ** -24) * v.abs())
    return out


def _close(name, got, ref):
    want, tol = ref
    assert got.shape == want.shape
    err = (got.double() - want).abs()
    assert (err <= tol + 1e-30).all(), f"{name}: {float((err / (tol + 1e-30)).max())} of its bound"


def _check(got, ref):
    for n, v in got.items():
        if v is not None:
            _close(n, v, ref[n])


def _run(x, W, b, r, dy, act):
    ws = LinearWorkspace(*x.shape, W.shape[1], act)
    y, z = linear_forward(x, W, b, r, act, for_backward=True, workspace=ws)
    dx, dW, db = linear_backward(dy, x, W, z, b, act, workspace=ws)
    assert ws.status() == 0
    return {"y": y, "dx": dx, "dW": dW, "dbias": db}


@pytest.mark.parametrize("T,K,N,act,bias,residual", [
    (1, 8, 8, "gelu", BF, True), (1, 72, 1000, None, F32, False), (2, 2048, 64, "silu", None, True),
    (8, 136, 264, "gelu_tanh", BF, True), (9, 1032, 72, "silu", F32, False), (16, 2048, 1416, "gelu", BF, True),
    (17, 264, 520, None, BF, True), (40, 1160, 712, "silu", BF, False), (100, 64, 64, "gelu", F32, True),
    (128, 2048, 2816, "gelu_tanh", BF, True), (129, 328, 200, None, None, True), (200, 4096, 256, "silu", BF, True),
    (256, 256, 256, None, None, False), (257, 264, 264, "gelu", BF, True), (300, 72, 2056, "silu", F32, False),
    (777, 1160, 712, "gelu", BF, True), (1000, 1000, 1000, "gelu_tanh", None, True), (2049, 136, 1032, None, F32, True),
    (4096, 512, 2816, "silu", BF, False), (130, 64, 7168, "gelu", F32, False), (10000, 64, 72, "silu", BF, True),
    (9000, 72, 264, None, BF, False), (300, 136, 5000, None, None, True), (5000, 520, 264, "gelu_tanh", F32, False),
])
def test_against_64_bits(T, K, N, act, bias, residual):
    inp = _inputs(T, K, N, T + K + N, bias, residual)
    _check(_run(*inp, act), _ref(*inp, act))


@pytest.mark.parametrize("T", [3, 60, 500])
def test_strided_rows(T):
    K, N = 264, 328
    x, W, b, r, dy = _inputs(T, K, N)
    wide = [torch.full((T, n + 24), float("nan"), device="cuda", dtype=BF) for n in (K, N, N)]
    xs, rs, ds = (w[:, 8: 8 + t.shape[1]].copy_(t) for w, t in zip(wide, (x, r, dy)))
    whole, cut = _run(x, W, b, r, dy, "silu"), _run(xs, W, b, rs, ds, "silu")
    for n in whole:
        assert torch.equal(whole[n], cut[n]), n
    with pytest.raises(B.MoeError):  # rows that no 16-byte copy starts at
        linear_forward(torch.empty(T, K + 4, device="cuda", dtype=BF)[:, :K], W)


def test_autograd_takes_any_layout():
    T, K, N = 37, 136, 72
    x, W, b, r, dy = _inputs(T, K, N)
    ref = _ref(x, W, b, r, dy, "gelu")
    flat = torch.empty(T * K + 1, device="cuda", dtype=BF)  # off every 16-byte boundary
    odd = flat[1:].view(T, K).copy_(x).requires_grad_()
    Wt = W.t().contiguous().t().requires_grad_()
    bb, rr = b.clone().requires_grad_(), r.clone().requires_grad_()
    y = linear(odd, Wt, bb, rr, "gelu")
    _close("y", y, ref["y"])
    gx, gW, gb, gr = torch.autograd.grad(y, (odd, Wt, bb, rr), dy)
    _check({"dx": gx, "dW": gW, "dbias": gb}, ref)
    assert torch.equal(gr, dy)
    # leading axes, gradient of a sum (its rows all one element), one input wanted
    x3 = x[:36].view(4, 9, K).requires_grad_()
    y3 = linear(x3, W, None, None, "silu")
    assert y3.shape == (4, 9, N)
    g3, = torch.autograd.grad(y3.sum(), x3)
    one = _ref(x[:36], W, None, None, torch.ones(36, N, device="cuda"), "silu")
    _close("dx", g3.view(36, K), one["dx"])
    with torch.no_grad():
        assert torch.equal(linear(x, W, b, r, "gelu"), y)


def test_each_gradient_alone():
    x, W, b, r, dy = _inputs(300, 264, 136)
    _, z = linear_forward(x, W, b, r, "gelu", for_backward=True)
    dx, dW, db = linear_backward(dy, x, W, z, b, "gelu")
    for want in ((True, False), (False, True), (False, False)):
        ex, eW, eb = linear_backward(dy, x, W, z, b, "gelu", want)
        assert (ex is None) != want[0] and (eW is None) != want[1]
        assert torch.equal(eb, db)
        assert ex is None or torch.equal(ex, dx)
        assert eW is None or torch.equal(eW, dW)
    ex, eW, eb = linear_backward(dy, x, W, z, None, "gelu")
    assert eb is None and torch.equal(ex, dx) and torch.equal(eW, dW)


@pytest.mark.parametrize("T,K,N,act", [(9000, 72, 264, None), (130, 64, 7168, "silu"), (6000, 64, 6000, None), (10000, 2048, 64, "gelu")])
def test_deep_gradients_alone(T, K, N, act):
    """Products whose K is split, by themselves and beside the other one, with strided rows,
    scratch filled before and not a byte of it behind its end touched."""
    x, W, b, r, dy = _inputs(T, K, N, 5, residual=False)
    x = torch.cat([x, x], 1)[:, :K]
    z = linear_forward(x, W, b, None, act, True)[1]
    ref = _ref(x, W, b, None, dy, act)
    s = B.linear_shape(T, K, N, act)
    n = B.moe_linear_workspace(s, True)
    for dx, dW, db in ((True, True, True), (True, False, False), (False, True, False), (True, True, False), (False, True, True)):
        ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
        ws[:4] = 0
        out = {"dx": torch.empty(T, K, device="cuda", dtype=BF) if dx else None, "dW": torch.empty(K, N, device="cuda", dtype=BF) if dW else None,
               "dbias": torch.empty_like(b) if db else None}
        B.moe_linear_backward(s, dy, x, W, z, ws, *out.values())
        assert (ws[n:] == 255).all() and not ws[:4].any()
        _check(out, ref)


@pytest.mark.parametrize("T", [5, 70, 600])
def test_residual_in_place(T):
    x, W, b, r, _ = _inputs(T, 264, 520)
    want, _ = linear_forward(x, W, b, r, "silu")
    s = B.linear_shape(T, 264, 520, "silu")
    ws = torch.empty(B.moe_linear_workspace(s, False), dtype=torch.uint8, device="cuda")
    B.moe_linear_forward(s, x, W, b, r, None, ws, r)
    assert torch.equal(r, want)


@pytest.mark.parametrize("act", [None, "silu", "gelu", "gelu_tanh"])
def test_wide_range_of_z(act):
    """Far tails, exact zeros: the products are exact, z runs over [-30, 30]."""
    K = N = 64
    x = torch.zeros(200, K, device="cuda")
    x[:, 0] = torch.linspace(-30, 30, 200, device="cuda")
    x, W = x.to(BF), torch.zeros(K, N, device="cuda", dtype=BF)
    W[0] = 1.0
    dy = torch.ones(200, N, device="cuda", dtype=BF)
    y, z = linear_forward(x, W, None, None, act, for_backward=True)
    dx, _, db = linear_backward(dy, x, W, z, torch.zeros(N, device="cuda"), act)
    v, s = _act(x[:, :1].double().expand(-1, N), act)
    # the argument of exp is up to 0.5 z^2 (gelu) or 0.08 z^3 (tanh), rounded at 2^-23 of itself before it
    zz = x[:, :1].double().abs()
    arg = 2.0 ** -22 * (1 + zz + zz * zz + 0.08 * zz ** 3)
    tiny = 2.0 ** -126
    assert ((y.double() - v).abs() <= (HALF + 2 * arg) * v.abs() + tiny * 32).all()
    # the fast divide gives 0 for divisors above 2^126 (its documented range): sigmoid errs by up to 2^-126 there, and
    # the slope by that times 1 + |z| 1.6 (1 + 0.135 z^2), the factor of sigmoid (1 - sigmoid) in the tanh form
    tiny = tiny * (1 + zz * 1.6 * (1 + 0.135 * zz * zz))
    # dx = 64 equal terms, each rounded to bf16, their sum rounded again; the slope's two terms cancel near its zero
    parts = s.abs() + (v.abs() * (1 + zz * zz) if act else 0)
    want = 64 * s[:, 0]
    assert ((dx[:, 0].double() - want).abs() <= 64 * ((HALF + A) * s.abs() + arg * parts + tiny)[:, 0] + HALF * want.abs()).all()
    assert ((db.double() - s.sum(0)).abs() <= (arg * parts + 264 * 2.0 ** -24 * s.abs() + tiny).sum(0)).all()


def test_nan_and_infinity_stay_in_their_row():
    for T in (8, 300):
        x, W, b, r, dy = _inputs(T, 136, 264)
        clean, _ = linear_forward(x, W, b, r, "silu")
        x[3, 5], r[5, 7] = float("nan"), float("inf")
        y, z = linear_forward(x, W, b, r, "silu", for_backward=True)
        rows = [i for i in range(T) if i not in (3, 5)]
        assert torch.equal(y[rows], clean[rows]) and y[3].isnan().all()
        assert y[5, 7] == float("inf") and torch.equal(y[5, 8:], clean[5, 8:])
        dx, _, _ = linear_backward(dy, x, W, z, None, "silu")
        assert dx[3].isnan().all() and dx[rows].isfinite().all()


def test_no_rows():
    W, b = torch.randn(64, 72, device="cuda").to(BF), torch.randn(72, device="cuda")
    x = torch.empty(0, 64, device="cuda", dtype=BF)
    y, z = linear_forward(x, W, b, None, "silu", for_backward=True)
    assert y.shape == (0, 72)
    dx, dW, db = linear_backward(y, x, W, z, b, "silu")
    assert dx.shape == (0, 64) and not dW.any() and not db.any()


def test_elements_past_32_bits():
    T, K, N, g = 300_001, 64, 7168, torch.Generator(device="cuda").manual_seed(3)
    assert T * N > 2 ** 31
    _, W, b, _, _ = _inputs(8, K, N)
    x, r, dy = (torch.empty(T, n, device="cuda", dtype=BF).normal_(generator=g) for n in (K, N, N))
    y, z = linear_forward(x, W, b, r, "silu", for_backward=True)
    dx, dW, db = linear_backward(dy, x, W, z, b, "silu")
    for at in (slice(0, 3), slice(T - 300, T)):
        ref = _ref(x[at], W, b, r[at], dy[at], "silu")
        _close("y", y[at], ref["y"])
        _close("dx", dx[at], ref["dx"])
    # some columns of dW: FP32 sums of T terms, 16 at a time, that may be cut instead of
    # rounded at each step: (T / 16 + 64) 2^-22 of the sum of their sizes
    cols = torch.cat([torch.arange(40, device="cuda"), torch.arange(N - 40, N, device="cuda")])
    ref = _ref(x, W[:, cols], b[cols], r[:, cols], dy[:, cols], "silu")
    size = x.double().abs().t() @ (dy[:, cols].double() * _act(z[:, cols].double(), "silu")[1]).abs()
    want, tol = ref["dW"]
    _close("dW", dW[:, cols], (want, tol + (T / 16 + 64) * 2.0 ** -22 * size))
    _close("dbias", db[cols], ref["dbias"])


def test_rows_behind_the_last_stay():
    for T in (5, 40, 300):
        x, W, b, r, dy = _inputs(T, 72, 136)
        s = B.linear_shape(T, 72, 136, "silu")
        ws = torch.empty(max(B.moe_linear_workspace(s, d) for d in (False, True)), dtype=torch.uint8, device="cuda")
        y, dx = (torch.full((T + 9, n), 7.0, device="cuda", dtype=BF) for n in (136, 72))
        z = torch.full((T + 9, 136), 7.0, device="cuda")
        dW, db = torch.full((72 + 1, 136), 7.0, device="cuda", dtype=BF), torch.full((137,), 7.0, device="cuda")
        B.moe_linear_forward(s, x, W, b, r, z, ws, y)
        B.moe_linear_backward(s, dy, x, W, z, ws, dx, dW, db)
        for t, n in ((y, T), (dx, T), (z, T), (dW, 72), (db, 136)):
            assert (t[n:] == 7.0).all()


@pytest.mark.parametrize("T", [8, 100, 600])
def test_graph_replay_and_streams(T):
    x, W, b, r, dy = _inputs(T, 264, 520)

    def step():
        y, z = linear_forward(x, W, b, r, "gelu", for_backward=True)
        return (y, *linear_backward(dy, x, W, z, b, "gelu"))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(want, again))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        for t in out:
            t.fill_(3.0)
        g.replay()
        assert all(torch.equal(a, c) for a, c in zip(want, out))
    x2 = _inputs(T, 264, 520, seed=9)[0]  # other inputs in the same buffers
    x.copy_(x2)
    g.replay()
    fresh = step()
    assert all(torch.equal(a, c) for a, c in zip(fresh, out))


def test_gradient_against_differences():
    """Directional differences of the definition in 64 bits, step 1e-4: their own error is of the order 1e-8."""
    T, K, N = 90, 72, 40
    x, W, b, r, dy = _inputs(T, K, N, bias=F32)
    for act in ("silu", "gelu", "gelu_tanh"):
        got = _run(x, W, b, r, dy, act)
        ref = _ref(x, W, b, r, dy, act)
        base = {"dx": x.double(), "dW": W.double(), "dbias": b.double()}
        for n, v in base.items():
            d = torch.randn(v.shape, device="cuda", dtype=torch.float64, generator=torch.Generator("cuda").manual_seed(3))

            def loss(h):
                m = {**base, n: v + h * d}
                return (_act(m["dx"] @ m["dW"] + m["dbias"], act)[0] * dy.double()).sum()

            diff = (loss(1e-4) - loss(-1e-4)) / 2e-4
            tol = (ref[n][1] * d.abs()).sum()  # the elements' bounds
            assert abs((got[n].double() * d).sum() - diff) <= tol + 1e-5 * abs(diff) + 1e-6


def test_second_order_raises():
    x, W, b, r, dy = _inputs(10, 64, 64)
    x.requires_grad_()
    g, = torch.autograd.grad(linear(x, W, b, r, "silu").float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()


def test_refusals():
    x, W, b, r, dy = _inputs(10, 64, 72)
    for bad in (lambda: linear_forward(x, W[:32]), lambda: linear_forward(x, W, b[:8]), lambda: linear_forward(x, W, b, r[:9]),
                lambda: linear_forward(x, W, activation="tanh"), lambda: linear(x, W, None, r[:1]),
                lambda: linear_backward(dy[:9], x, W), lambda: linear_backward(dy, x, W, None, None, "silu"),
                lambda: linear_forward(x, W, workspace=LinearWorkspace(11, 64, 72))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: linear_forward(x.float(), W), lambda: linear_forward(x, W.half()), lambda: linear_forward(x, W, b.half()),
                lambda: linear_forward(x.cpu(), W.cpu()), lambda: linear_forward(x, W, b, r.float())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(B.MoeError):
        linear_forward(x[:, :60], W[:60])
