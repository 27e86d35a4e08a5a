"""The joint between two halves of a block against 64 bits.

Tolerances, element by element, carried through the formulas.  An FP32 sum over
a row adds in a tree no deeper than 30 and H / 1024 terms of one thread: g = (30
+ H / 1024) 2^-24 of the sum of the terms' sizes; a sum over the rows is no
deeper than rows / 100 + 64.  An error e_v of the values moves the mean by mean
e_v + g mean|v| and 1 / sqrt(var) by half of var's relative error, 2 mean(|d|
(e_v + e_mean)) / var + g + 2^-22, and rsqrtf errs by 2^-22 more.  Every other
operation rounds at 2^-24 of its result (a few of them together: 2^-22 of the
terms' sizes).  Outputs are rounded once, by at most half a step: eps / 2 of
their type, and below the smallest normal number by half the spacing there."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import residual_norm, residual_norm_backward, residual_norm_forward

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAMES = ("dout", "dresidual", "dweight", "dbias", "dpost_weight", "dpost_bias", "dgate")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


def _case(rows, H, t=BF, wt=F32, bias=True, post=True, post_bias=True, gate="channel", alpha=0.5, kind="layer", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows + H)

    def n(shape, std, dt, at=0.0):
        return (at + torch.randn(shape, generator=g, device="cuda") * std).to(dt)

    r = n((rows, H), 1.0, F32)
    r[:, :: max(1, H // 4)] *= 8.0
    r = r * (0.5 + torch.rand((rows, 1), generator=g, device="cuda")) + n((rows, 1), 0.3, F32)
    return dict(out=n((rows, H), 0.7, t), residual=r.to(t), weight=n((H,), 0.2, wt, 1.0), bias=n((H,), 0.1, wt) if bias else None,
                post_weight=n((H,), 0.2, wt, 1.0) if post else None, post_bias=n((H,), 0.1, wt) if post and post_bias else None,
                gate={"none": None, "channel": n((H,), 0.2, wt, 0.5), "token": n((rows, 1), 0.5, wt)}[gate],
                residual_scale=alpha, kind=kind), n((rows, H), 1.0, t), n((rows, H), 1.0, t)


def _ref(c, ds, dn, eps=1e-5):
    """{name: (value, tolerance before the last rounding)} in 64 bits."""
    o, r, w, b, pw, pb, gate = (None if c[k] is None else c[k].double() for k in
                                ("out", "residual", "weight", "bias", "post_weight", "post_bias", "gate"))
    rows, H = o.shape
    layer, alpha = c["kind"] == "layer", c["residual_scale"]
    g, gc, u24, u22 = (30 + H / 1024) * 2.0 ** -24, (rows / 100 + 64) * 2.0 ** -24, 2.0 ** -24, 2.0 ** -22

    def mean(v):
        return v.mean(1, True)

    def norm(v, ev):
        """(z, its error, 1 / sqrt, its relative error)"""
        m = mean(v) if layer else torch.zeros_like(v[:, :1])
        em = mean(ev) + g * mean(v.abs()) if layer else 0.0 * m
        d = v - m
        ed = ev + em + u24 * (v.abs() + m.abs())
        var = mean(d * d) + eps
        rs = var.rsqrt()
        er = mean(2 * d.abs() * ed) / var / 2 + g + 2 * u22
        return d * rs, rs * ed + (d * rs).abs() * (er + u24), rs, er

    def norm_grad(p, ep, z, ez, rs, er):
        """(gradient through z of p, its error)"""
        m1, m2 = mean(p) if layer else 0.0 * rs, mean(p * z)
        e1 = mean(ep) + g * mean(p.abs()) if layer else 0.0
        e2 = mean(ep * z.abs() + p.abs() * ez) + g * mean((p * z).abs())
        size = p.abs() + m1.abs() + (z * m2).abs()
        return rs * (p - m1 - z * m2), rs * (ep + e1 + ez * m2.abs() + z.abs() * e2 + u22 * size + er * size)

    zero = torch.zeros_like(o)
    if pw is None:
        u, eu, oz, eoz = o, zero, o, zero
    else:
        oz, eoz, ors, eor = norm(o, zero)
        pbv = 0 * pw if pb is None else pb
        u = oz * pw + pbv
        eu = eoz * pw.abs() + u22 * ((oz * pw).abs() + pbv.abs())
    gv = torch.ones(1, device="cuda", dtype=torch.float64) if gate is None else gate
    s = alpha * r + gv * u
    es = gv.abs() * eu + u22 * ((alpha * r).abs() + (gv * u).abs())
    z, ez, rs, er = norm(s, es)
    bv = 0 * w if b is None else b
    ref = {"stream": (s, es), "normed": (z * w + bv, ez * w.abs() + u22 * ((z * w).abs() + bv.abs()))}
    if ds is None and dn is None:
        return ref
    ds, dn = (zero if v is None else v.double() for v in (ds, dn))
    h = dn * w
    a, ea = norm_grad(h, u24 * h.abs(), z, ez, rs, er)
    D, eD = ds + a, ea + u24 * (ds.abs() + a.abs())
    ref["dresidual"] = alpha * D, abs(alpha) * eD + u24 * (alpha * D).abs()
    q, eq = gv * D, gv.abs() * eD + u24 * (gv * D).abs()
    if pw is None:
        ref["dout"] = q, eq
    else:
        ref["dout"] = norm_grad(q * pw, eq * pw.abs() + u24 * (q * pw).abs(), oz, eoz, ors, eor)

    def rowsum(v, ev):
        return v.sum(0), ev.sum(0) + gc * v.abs().sum(0)

    ref["dweight"] = rowsum(dn * z, dn.abs() * ez)
    if b is not None:
        ref["dbias"] = rowsum(dn, zero)
    if pw is not None:
        ref["dpost_weight"] = rowsum(q * oz, eq * oz.abs() + q.abs() * eoz)
    if pb is not None:
        ref["dpost_bias"] = rowsum(q, eq)
    if gate is not None and gate.dim() == 1:
        A, eA = rowsum(D * oz, eD * oz.abs() + D.abs() * eoz)
        C, eC = rowsum(D, eD)
        p1, p0 = (1.0 + 0 * A, 0.0 * A) if pw is None else (pw, 0 * pw if pb is None else pb)
        ref["dgate"] = p1 * A + p0 * C, p1.abs() * eA + p0.abs() * eC + u22 * ((p1 * A).abs() + (p0 * C).abs())
    elif gate is not None:
        v = D * u
        ref["dgate"] = v.sum(1, True), (eD * u.abs() + D.abs() * eu).sum(1, True) + (g + u22) * v.abs().sum(1, True)
    return ref


def _half(t):
    return torch.finfo(t).eps / 2


def _close(name, got, ref):
    want, tol = ref
    assert got.shape == want.shape, name
    low = {BF: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}[got.dtype]  # half the spacing of the subnormal numbers
    tol = tol + _half(got.dtype) * (want.abs() + tol) + low
    err = (got.double() - want).abs()
    assert (err <= tol).all(), f"{name}: {float((err / tol).max())} of its bound"


def _run(c, ds, dn):
    stream, normed, stats = residual_norm_forward(**c)
    bwd = {k: v for k, v in c.items() if k not in ("out", "residual", "weight")}
    grads = residual_norm_backward(ds, dn, c["out"], c["residual"], c["weight"], stats, **bwd)
    return {"stream": stream, "normed": normed, **{n: v for n, v in zip(NAMES, grads) if v is not None}}


def _check(c, ds, dn):
    got, ref = _run(c, ds, dn), _ref(c, ds, dn)
    assert set(got) == set(ref)
    for n, v in got.items():
        _close(n, v, ref[n])
    return got


@pytest.mark.parametrize("rows,H,options", [
    (1, 1, dict(kind="rms")), (1, 8, dict()), (3, 7, dict(gate="token")), (5, 64, dict(t=F32)), (64, 128, dict(t=F32)),
    (2, 33, dict(t=F16, wt=F16)), (300, 64, dict(kind="rms", gate="none", post=False)), (500, 250, dict(wt=BF)),
    (1000, 256, dict(gate="token", post_bias=False)), (31, 257, dict(kind="rms", bias=False)),
    (700, 1001, dict(t=F16, alpha=1.25)), (400, 1024, dict(t=F32, kind="rms", post=False)),
    (3000, 512, dict(gate="channel", post=False)), (17, 264, dict()), (85, 1000, dict(t=F16)), (168, 1024, dict(wt=BF)),
    (9, 2048, dict(gate="token")), (24, 3000, dict(t=F32)), (700, 33, dict(t=F16, wt=F16)), (2, 7168, dict()), (640, 2048, dict(kind="rms", gate="none", post=False, bias=False)),
    (333, 2049, dict(gate="token")), (200, 4100, dict(t=F32, gate="channel")), (170, 7161, dict(kind="rms", gate="token")),
    (200, 7168, dict(wt=BF)), (160, 7168, dict(t=F32, gate="token")), (20, 7169, dict(t=F16)), (9, 10000, dict(gate="token")),
    (400, 9000, dict(kind="rms", post=False)), (3, 40000, dict(t=F32, gate="channel", wt=F32)), (152, 7168, dict(post=False)),
])
def test_against_64_bits(rows, H, options):
    _check(*_case(rows, H, **options))


@pytest.mark.parametrize("t,wt", [(BF, BF), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_every_form(t, wt, kind, gate):
    for H in (96, 91):
        for post, post_bias, bias in ((False, False, False), (True, False, True), (True, True, False)):
            _check(*_case(77, H, t, wt, bias, post, post_bias, gate, 1.0, kind))


@pytest.mark.parametrize("H", [64, 72, 333, 8000])
def test_one_gradient_alone(H):
    c, ds, dn = _case(40, H)
    _check(c, ds, None)
    _check(c, None, dn)


@pytest.mark.parametrize("H", [128, 130, 7300])
def test_strided_rows(H):
    c, ds, dn = _case(50, H, gate="token")
    whole = _run(c, ds, dn)
    for pad in (16, 3):  # on 16-byte boundaries, off them
        def wide(t):
            return torch.full((50, H + pad), float("nan"), device="cuda", dtype=t.dtype)[:, :H].copy_(t)

        cut = _run({**c, "out": wide(c["out"]), "residual": wide(c["residual"])}, wide(ds), wide(dn))
        for n in whole:
            # the columns a thread takes, and so the order of sums, go by the rows' alignment
            assert torch.equal(whole[n], cut[n]) or (pad == 3 and torch.allclose(whole[n].float(), cut[n].float(), 0.02, 0.02)), n
        for n, v in cut.items():
            _close(n, v, _ref(c, ds, dn)[n])


def test_last_rows_and_columns_stay():
    for H in (64, 61, 7200):
        rows = 30
        c, ds, dn = _case(rows, H, gate="token")
        s = B.residual_norm_shape(rows, H, BF, F32, "layer", B.GATE_TOKEN, 0.5)
        buf = {n: torch.full((rows * H + 40,), 7.0, device="cuda", dtype=BF) for n in ("stream", "normed", "dout", "dres")}
        par = [torch.full((H + 40,), 7.0, device="cuda") for _ in range(4)]
        dg, stats = torch.full((rows + 9,), 7.0, device="cuda"), torch.full((4 * rows + 9,), 7.0, device="cuda")
        ws = torch.empty(B.moe_residual_norm_workspace(s), dtype=torch.uint8, device="cuda")
        p = [c[k] for k in ("gate", "post_weight", "post_bias", "weight")]
        B.moe_residual_norm_forward(s, c["out"], c["residual"], *p, c["bias"], buf["stream"], buf["normed"], stats)
        B.moe_residual_norm_backward(s, ds, dn, c["out"], c["residual"], *p, stats, ws, buf["dout"], buf["dres"], *par, dg)
        assert all((t[rows * H:] == 7.0).all() for t in buf.values()) and all((t[H:] == 7.0).all() for t in par)
        assert (dg[rows:] == 7.0).all() and (stats[4 * rows:] == 7.0).all()


@pytest.mark.parametrize("H", [64, 65, 8001])
def test_in_place(H):
    c, _, _ = _case(33, H)
    want = residual_norm_forward(**c)
    s = B.residual_norm_shape(33, H, BF, F32, "layer", B.GATE_CHANNEL, 0.5)
    r, normed, stats = c["residual"].clone(), torch.empty_like(c["out"]), torch.empty(4, 33, device="cuda")
    B.moe_residual_norm_forward(s, c["out"], r, c["gate"], c["post_weight"], c["post_bias"], c["weight"], c["bias"], r, normed, stats)
    assert torch.equal(r, want[0]) and torch.equal(normed, want[1])


@pytest.mark.parametrize("H", [96, 97, 7500])
def test_bad_rows_stay_apart(H):
    c, ds, dn = _case(20, H, gate="none")
    clean = _run(c, ds, dn)
    c["residual"][3, 5], c["out"][7, 1], dn[11, 2] = float("nan"), float("inf"), float("nan")
    got = _run(c, ds, dn)
    ok = [i for i in range(20) if i not in (3, 7, 11)]
    for n in ("stream", "normed", "dout", "dresidual"):
        assert torch.equal(got[n][ok], clean[n][ok]), n
    assert got["normed"][3].isnan().all() and got["normed"][7].isnan().all() and got["dout"][11].isnan().all()
    assert torch.equal(got["normed"][11], clean["normed"][11])


def test_constant_rows():
    """A variance of zero: 1 / sqrt(eps), and rows of zeros."""
    for H in (64, 63):
        c, ds, dn = _case(6, H, gate="none", post=False)
        c["out"][:3], c["residual"][:3] = 1.0, 2.0
        c["out"][4], c["residual"][4] = 0.0, 0.0
        _check(c, ds, dn)


@pytest.mark.parametrize("H", [7168, 7161])
def test_elements_past_32_bits(H):
    rows, g = 300_001, torch.Generator(device="cuda").manual_seed(3)  # 300001 x 7161 > 2^31
    assert rows * H > 2 ** 31
    c = _case(8, H, gate="channel", kind="rms")[0]
    c["out"], c["residual"], ds, dn = (torch.empty(rows, H, device="cuda", dtype=BF).normal_(generator=g) for _ in range(4))
    stream, normed, stats = residual_norm_forward(**c)
    bwd = {k: v for k, v in c.items() if k not in ("out", "residual", "weight")}
    grads = residual_norm_backward(ds, dn, c["out"], c["residual"], c["weight"], stats, **bwd)
    for at in (slice(0, 3), slice(rows - 400, rows)):
        ref = _ref(dict(c, out=c["out"][at], residual=c["residual"][at]), ds[at], dn[at])
        for n, v in (("stream", stream), ("normed", normed), ("dout", grads[0]), ("dresidual", grads[1])):
            _close(n, v[at], ref[n])


def test_no_rows():
    c, ds, dn = _case(0, 64)
    got = _run(c, ds, dn)
    assert got["stream"].shape == (0, 64)
    for n in NAMES[2:]:
        assert not got[n].any()


@pytest.mark.parametrize("rows,H", [(300, 256), (70, 333), (5, 9000)])
def test_graph_replay_and_streams(rows, H):
    c, ds, dn = _case(rows, H, gate="token")
    want = _run(c, ds, dn)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = _run(c, ds, dn)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(want[n], again[n]) for n in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _run(c, ds, dn)
    for _ in range(3):
        for v in out.values():
            v.fill_(5.0)
        g.replay()
        assert all(torch.equal(want[n], out[n]) for n in want)


def test_autograd():
    c, ds, dn = _case(24, 80, gate="token")
    ref = _ref(c, ds, dn)
    shape = (2, 3, 4)
    leaf = {k: (v.view(*shape, -1) if k in ("out", "residual", "gate") else v).clone().requires_grad_()
            for k, v in c.items() if torch.is_tensor(v)}
    stream, normed = residual_norm(**leaf, residual_scale=0.5)
    assert stream.shape == normed.shape == (*shape, 80)
    _close("stream", stream.view(24, 80), ref["stream"])
    grads = torch.autograd.grad((stream, normed), list(leaf.values()), (ds.view(*shape, 80), dn.view(*shape, 80)))
    for (k, v), d in zip(leaf.items(), grads):
        assert d.shape == v.shape and d.dtype == v.dtype
        _close("d" + k, d.view(24, -1) if k in ("out", "residual", "gate") else d, ref["d" + k])
    # one output alone, with a gradient that is one number
    stream, normed = residual_norm(**leaf, residual_scale=0.5)
    d, = torch.autograd.grad(normed.sum(), leaf["out"])
    _close("dout", d.view(24, 80), _ref(c, None, torch.ones_like(dn))["dout"])
    stream, normed = residual_norm(**leaf, residual_scale=0.5)
    d, = torch.autograd.grad(normed.float().sum(), leaf["out"], create_graph=True)
    with pytest.raises(RuntimeError):
        d.float().sum().backward()
    # the same tensor as output and residual
    x = c["out"].clone().requires_grad_()
    stream, normed = residual_norm(x, x, c["weight"], kind="rms")
    d, = torch.autograd.grad((stream, normed), x, (ds, dn))
    one = _ref(dict(c, residual=c["out"], bias=None, post_weight=None, post_bias=None, gate=None, residual_scale=1.0, kind="rms"), ds, dn)
    want, tol = one["dout"]
    # the two gradients are rounded, added and rounded again
    assert ((d.double() - 2 * want).abs() <= 2 * tol + 2 * 2 * _half(BF) * (want.abs() + tol) + 1e-30).all()


def test_gradient_against_differences():
    """Directional differences of the definition in 64 bits."""
    for kind in ("layer", "rms"):
        for gate in ("channel", "token"):
            c, ds, dn = _case(12, 40, F32, gate=gate, kind=kind)
            got, ref = _run(c, ds, dn), _ref(c, ds, dn)
            names = [k for k, v in c.items() if torch.is_tensor(v)]

            def loss(**moved):
                v = _ref({**{k: c[k].double() if torch.is_tensor(c[k]) else c[k] for k in c}, **moved}, None, None)
                return (v["stream"][0] * ds.double()).sum() + (v["normed"][0] * dn.double()).sum()

            for k in names:
                d = torch.randn(c[k].shape, device="cuda", dtype=torch.float64, generator=torch.Generator("cuda").manual_seed(7))
                diff = (loss(**{k: c[k].double() + 1e-5 * d}) - loss(**{k: c[k].double() - 1e-5 * d})) / 2e-5
                tol = ((ref["d" + k][1] + 2.0 ** -24 * ref["d" + k][0].abs()) * d.abs()).sum()
                assert abs((got["d" + k].double() * d).sum() - diff) <= tol + 1e-6 * abs(diff) + 1e-6, k


def test_refusals():
    c, ds, dn = _case(10, 64)
    stats = residual_norm_forward(**c)[2]
    for bad in (dict(residual=c["residual"][:9]), dict(weight=c["weight"][:63]), dict(gate=c["gate"][:5]), dict(kind="batch"),
                dict(post_weight=None), dict(gate=torch.ones(10, 2, device="cuda"))):
        with pytest.raises(ValueError):
            residual_norm_forward(**{**c, **bad})
    for bad in (dict(residual=c["residual"].float()), dict(bias=c["bias"].to(BF)), dict(gate=c["gate"].half()),
                dict(weight=c["weight"].double()), dict(out=c["out"].cpu())):
        with pytest.raises(TypeError):
            residual_norm_forward(**{**c, **bad})
    for bad in (dict(weight=c["weight"].half(), bias=None, post_weight=None, post_bias=None, gate=None),
                dict(residual_scale=float("inf")), dict(eps=-1.0)):
        with pytest.raises(B.MoeError):
            residual_norm_forward(**{**c, **bad})
    with pytest.raises(ValueError):
        residual_norm_backward(ds[:9], dn, c["out"], c["residual"], c["weight"], stats)
    with pytest.raises(ValueError):
        residual_norm_backward(ds, dn, c["out"], c["residual"], c["weight"], stats[:, :9])
    with pytest.raises(ValueError):
        residual_norm(c["out"], c["residual"], c["weight"], gate=torch.ones(5, 1, device="cuda"))
    with pytest.raises(ValueError):  # a number is no gate, a single row's neither
        residual_norm(c["out"][:1], c["residual"][:1], c["weight"], gate=torch.tensor(1.0, device="cuda"))
