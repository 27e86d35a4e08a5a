"""Layer norm forward and backward against the formula in 64 bits.

Tolerances, u = 2^-24 (f32), ut = the output type's half spacing (2^-9 bf16,
2^-12 f16 relative to the value rounded up to 2^-8 / 2^-11; f32: u).
Forward, per element: the mean's error is at most ~64 u max|x| (partial sums
of at most 64 terms per thread, then trees), and z = (x - m) s carries it times
s; so |err| <= (ut + 16 u) |y| + 128 u s max|x| |w|.
dx, per element: one rounding of the output plus FP32 sums of H terms of the
size of |g| and |g z|: (ut + 32 u)|dx| + 128 u s (|g| + mean|g| + |z| mean|g z|
+ s max|x| (mean |g z| + |z| mean|g|)).
dweight, dbias: (2 ut_w + 2 sqrt(rows) u ...) bounded by 128 u sum |dy z|
(+ the mean's error times sum |dy|) plus the rounding to weight's type."""
import numpy as np
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import layer_norm, layer_norm_backward, layer_norm_forward

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UT = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


def _ref(x, w, b, eps, dy=None):
    x, w = x.double(), w.double()
    m = x.mean(1, keepdim=True)
    s = 1.0 / torch.sqrt((x - m).square().mean(1, keepdim=True) + eps)
    z = (x - m) * s
    out = dict(m=m, s=s, z=z, y=z * w + (0 if b is None else b.double()))
    if dy is not None:
        dy = dy.double()
        g = dy * w
        out.update(g=g, dx=s * (g - g.mean(1, keepdim=True) - z * (g * z).mean(1, keepdim=True)),
                   dw=(dy * z).sum(0), db=dy.sum(0), adw=(dy * z).abs().sum(0), adb=dy.abs().sum(0))
    return out


def _close(got, want, tol, name):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} off, worst {float((err / tol.clamp_min(1e-300)).max()):.2f} of its bound"


def _inputs(rows, H, t, wt, bias, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, H + pad, generator=g) * (0.5 + torch.rand(rows, 1, generator=g)) + torch.randn(rows, 1, generator=g)
    dy = torch.randn(rows, H + pad, generator=g)
    w = 1 + 0.3 * torch.randn(H, generator=g)
    b = 0.2 * torch.randn(H, generator=g) if bias else None
    x, dy, w = x.to(t).cuda()[:, :H], dy.to(t).cuda()[:, :H], w.to(wt).cuda()
    return x, dy, w, (b.to(wt).cuda() if bias else None)


def _check(x, dy, w, b, eps=1e-5):
    t, wt = x.dtype, w.dtype
    y, mean, rstd = layer_norm_forward(x, w, b, eps)
    dx, dw, db = layer_norm_backward(dy, x, w, mean, rstd, b is not None)
    r = _ref(x, w, b, eps, dy)
    rows, H = x.shape
    mx = x.double().abs().amax(1, keepdim=True)
    ym = 128 * U * r["s"] * mx  # error of z through the mean and the statistics
    wa = w.double().abs()
    _close(y, r["y"], (UT[t] + 16 * U) * r["y"].abs() + ym * wa + 64 * U * (r["z"].abs() * wa), "y")
    ag, agz = r["g"].abs().mean(1, keepdim=True), (r["g"] * r["z"]).abs().mean(1, keepdim=True)
    tol = (UT[t] + 32 * U) * r["dx"].abs() + 128 * U * r["s"] * (r["g"].abs() + ag + r["z"].abs() * agz)
    _close(dx, r["dx"], tol + r["s"] * ym * (agz + r["z"].abs() * ag), "dx")
    _close(dw, r["dw"], UT[wt] * r["dw"].abs() + 128 * U * r["adw"] + (ym * dy.double().abs()).sum(0), "dweight")
    if b is not None:
        _close(db, r["db"], UT[wt] * r["db"].abs() + 128 * U * r["adb"], "dbias")
    else:
        assert db is None
    return y, dx, dw, db


@pytest.mark.parametrize("rows,H,t,wt,bias", [
    (1, 1, F32, F32, True), (1, 64, BF, BF, True), (3, 7, F32, F32, False), (64, 128, F32, F32, True),
    (130, 1000, BF, F32, True), (5, 1001, F16, F32, False), (257, 1024, BF, F32, True), (33, 1032, F16, F16, True),
    (700, 2048, BF, F32, True), (9, 2049, BF, BF, True), (310, 7168, BF, F32, True), (611, 333, F32, F32, True),
    (20, 8192, F16, F32, True), (7, 8200, BF, F32, True), (5, 8191, F32, F32, True), (4, 16384, BF, BF, False),
    (4, 16392, BF, F32, True), (3, 20001, F16, F32, True), (2, 40000, F32, F32, True), (1300, 96, BF, F32, True),
])
def test_against_64_bits(rows, H, t, wt, bias):
    _check(*_inputs(rows, H, t, wt, bias, seed=rows * 31 + H))


@pytest.mark.parametrize("rows,H,t,wt,bias,pad", [
    (8001, 33, BF, F32, True, 0), (7700, 333, F32, F32, False, 0), (7400, 1001, F16, F16, True, 0),
    (7400, 250, BF, BF, False, 8), (2600, 2047, F32, F32, True, 0), (1500, 5003, BF, F32, True, 0),
    (1400, 5002, BF, F32, False, 16), (1000, 10001, F16, F32, True, 0), (950, 7161, F32, F32, True, 0),
])
def test_many_rows_between_vector_boundaries(rows, H, t, wt, bias, pad):
    """Widths that 16 bytes do not divide, enough rows for persistent blocks: rows start anywhere in a vector, the last
    one's vector ends past the tensor."""
    x, dy, w, b = _inputs(rows, H, t, wt, bias, seed=H, pad=pad)
    if not pad:  # nothing behind the last row is read into a result or written
        es = x.element_size()
        buf = torch.full((rows * H + 64 // es,), float("nan"), dtype=t, device="cuda")
        buf[: rows * H] = x.flatten()
        x = buf[: rows * H].view(rows, H)
    _check(x, dy, w, b)


@pytest.mark.parametrize("pad", [1, 8])
def test_strided_rows(pad):
    x, dy, w, b = _inputs(77, 520, BF, F32, True, 5, pad=pad)
    assert x.stride(0) == 520 + pad
    _check(x, dy, w, b)


def test_unaligned_base():
    buf = torch.randn(40 * 256 + 1, dtype=F32).to(BF).cuda()
    x = buf[1:].view(40, 256)
    _, dy, w, b = _inputs(40, 256, BF, F32, True, 6)
    _check(x, dy, w, b)


def test_large_offset_and_constant_rows():
    """Rows far from zero lose nothing to cancellation; a constant row has variance 0."""
    x, dy, w, b = _inputs(16, 512, F32, F32, True, 7)
    x = x + 1000.0
    x[3] = 2.5
    y, dx, _, _ = _check(x, dy, w, b)
    assert torch.equal(y[3], b) and torch.isfinite(dx).all()


def test_non_finite_rows_stay_in_their_row():
    x, dy, w, b = _inputs(6, 300, BF, F32, True, 8)
    good, *_ = layer_norm_forward(x, w, b)
    x[1, 7] = float("nan")
    x[4, 0] = float("inf")
    y, mean, rstd = layer_norm_forward(x, w, b)
    dx, dw, _ = layer_norm_backward(dy, x, w, mean, rstd)
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], good[keep]) and y[[1, 4]].isnan().all()
    assert torch.isfinite(dx[keep]).all() and dx[[1, 4]].isnan().all() and dw.isnan().all()


def test_no_rows():
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    y, mean, rstd = layer_norm_forward(x, w, w)
    dx, dw, db = layer_norm_backward(x, x, w, mean, rstd)
    assert y.shape == dx.shape == (0, 64) and not dw.any() and not db.any()


def test_gradient_against_differences():
    """d/dt of sum(dy y) along a direction, by central differences in 64 bits of the formula's forward."""
    x, dy, w, b = _inputs(4, 37, F32, F32, True, 9)
    xr, wr, br = x.clone().requires_grad_(), w.clone().requires_grad_(), b.clone().requires_grad_()
    layer_norm(xr, wr, br).backward(dy)
    h = 1e-5
    for t, grad, args in ((x, xr.grad, 0), (w, wr.grad, 1), (b, br.grad, 2)):
        d = torch.randn(t.shape, generator=torch.Generator().manual_seed(args)).double().cuda()
        at = [x.double(), w.double(), b.double()]
        vals = []
        for sgn in (1, -1):
            v = list(at)
            v[args] = at[args] + sgn * h * d
            vals.append((_ref(v[0], v[1], v[2], 1e-5)["y"] * dy.double()).sum())
        want = (vals[0] - vals[1]) / (2 * h)
        got = (grad.double() * d).sum()
        # the difference quotient is good to ~h^2 and 1e-16 / h; FP32 sums of 148 terms of size ~1
        assert abs(float(got - want)) <= 1e-6 * float((grad.double() * d).abs().sum()) + 1e-7


def test_leading_axes_transposed_input_and_other_stream():
    base = torch.randn(48, 5, 6, device="cuda")
    x = base.permute(1, 2, 0).requires_grad_()  # last axis not contiguous
    w = torch.rand(48, device="cuda").requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = layer_norm(x, w)
        y.sum().backward()
    torch.cuda.current_stream().wait_stream(s)
    assert y.shape == (5, 6, 48) and x.grad.shape == x.shape
    r = _ref(x.detach().reshape(30, 48), w.detach(), None, 1e-5, torch.ones(30, 48, device="cuda"))
    _close(y.detach().reshape(30, 48), r["y"], 1e-5 * (1 + r["y"].abs()), "y")
    _close(w.grad, r["dw"], 128 * U * (r["adw"] + 30 * 5), "dweight")


def test_deterministic():
    x, dy, w, b = _inputs(2000, 768, BF, F32, True, 10)
    a = _check(x, dy, w, b)
    c = _check(x, dy, w, b)
    for p, q in zip(a, c):
        assert torch.equal(p, q)


def test_refusals():
    x = torch.zeros(4, 16, dtype=BF, device="cuda")
    w = torch.ones(16, device="cuda")
    with pytest.raises(TypeError):
        layer_norm_forward(x.cpu(), w)
    with pytest.raises(TypeError):
        layer_norm_forward(x.double(), w)
    with pytest.raises(ValueError):
        layer_norm_forward(x, w[:8])
    with pytest.raises(TypeError):
        layer_norm_forward(x, w, torch.ones(16, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        layer_norm_forward(x.t(), torch.ones(4, device="cuda"))
    with pytest.raises(B.MoeError):
        layer_norm_forward(x, w, None, float("nan"))
    with pytest.raises(B.MoeError):
        layer_norm_forward(x, w.half())
    y, mean, rstd = layer_norm_forward(x, w)
    with pytest.raises(TypeError):
        layer_norm_backward(y.float(), x, w, mean, rstd)
    with pytest.raises(ValueError):
        layer_norm_backward(y[:2], x, w, mean, rstd)
