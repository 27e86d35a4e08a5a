"""The whole expert layer of decoding against 64 bits.

Routing first: the logits' FP32 sums err by at most (H / 512 + 22) 2^-24 of the sum
of the products' sizes (a thread's own terms, then a tree of 3 + 8 + 8 + rounding
steps), so where the k-th and the next logit are further apart than twice that the
choice has to be the one in 64 bits, and its weights differ by at most that error
times twice their size and a few roundings of 2^-22.

Then the layer for the routing that the kernel took, element by element.  An FP32
accumulation of K bf16 products in groups of 16 (and up to 16 ranges added after)
errs by at most A = 2^-19 of the sum of the products' sizes for the K used here.
The activation a (slope of silu at most 1.1, device exp 2^-18 of a) is rounded to
bf16 once: half a step, 2^-8 of it.  y is a sum of at most k + 1 terms in FP32 (2^-20
of their sizes) and is rounded once."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.layer import DecodeLayer, MoEWorkspace, moe_layer

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
A, HALF = 2.0 ** -19, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


def _weights(H, I, E, Is=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)

    return (n(H, E, std=H ** -0.5), n(E, H, 2 * I, std=H ** -0.5), n(E, I, H, std=I ** -0.5),
            n(H, 2 * Is, std=H ** -0.5) if Is else None, n(Is, H, std=Is ** -0.5) if Is else None)


def _x(T, H, seed=1):
    return torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF)


def _expert(x, W1, W2, c):
    """(value, tolerance before the last rounding) of one expert's output."""
    x, W1, W2 = x.double(), W1.double(), W2.double()
    h, eh = x @ W1, A * (x.abs() @ W1.abs())
    g, u = h.chunk(2, 1)
    eg, eu = eh.chunk(2, 1)
    if c > 0:
        g, u = g.clamp(-c, c), u.clamp(-c, c)
    s = g * torch.sigmoid(g)
    a = s * u
    ea = 1.1 * eg * u.abs() + s.abs() * eu + (HALF + 2.0 ** -18) * a.abs()
    return a @ W2, (ea + A * a.abs()) @ W2.abs()


def _check_layer(y, x, idx, w, W1, W2, S1, S2, c=0.0):
    E = W1.shape[0]
    want, tol, size = (torch.zeros(y.shape, dtype=torch.float64, device="cuda") for _ in range(3))
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if not len(t):
            continue
        v, ev = _expert(x[t], W1[e], W2[e], c)
        ww = w[t, j].double()[:, None]
        want.index_add_(0, t, ww * v)
        tol.index_add_(0, t, ww.abs() * ev)
        size.index_add_(0, t, (ww * v).abs())
    if S1 is not None:
        v, ev = _expert(x, S1, S2, c)
        want, tol, size = want + v, tol + ev, size + v.abs()
    err = (y.double() - want).abs()
    bound = tol + 2.0 ** -20 * size + HALF * (want.abs() + tol) + 1e-30
    assert (err <= bound).all(), f"{float((err / bound).max())} of its bound"


def _check_routing(x, router, idx, w, k):
    T, E = x.shape[0], router.shape[1]
    l = x.double() @ router.double()
    el = (x.shape[1] / 512 + 22) * 2.0 ** -24 * (x.double().abs() @ router.double().abs())
    top, order = torch.sort(l, dim=1, descending=True, stable=True)
    assert ((idx >= 0) & (idx < E)).all()
    for t in range(T):
        for j in range(k):
            a, b = int(idx[t, j]), int(order[t, j])
            # the same expert, or one whose logit is that near
            assert a == b or abs(float(l[t, a] - l[t, b])) <= 2 * float(el[t].max()), (t, j)
        assert len(set(idx[t].tolist())) == k
    chosen = torch.gather(l, 1, idx.long())
    want = torch.softmax(chosen, 1)
    assert ((w.double() - want).abs() <= want * (2 * el.max(1, keepdim=True).values + 2.0 ** -20 * (1 + chosen.abs().max()))).all()


def _run(T, H, I, E, k, Is=0, c=0.0, seed=0):
    router, W1, W2, S1, S2 = _weights(H, I, E, Is, seed)
    x = _x(T, H, seed + 1)
    layer = DecodeLayer(router, W1, W2, k, S1, S2, activation_clamp=c)
    y, idx, w = layer(x, return_routing=True)
    _check_routing(x, router, idx, w, k)
    _check_layer(y, x, idx, w, W1, W2, S1, S2, c)
    return layer, x, y


@pytest.mark.parametrize("T,H,I,E,k,Is", [
    (1, 64, 64, 1, 1, 0), (1, 128, 64, 8, 2, 0), (4, 128, 64, 8, 2, 64), (1, 2048, 1408, 64, 6, 2816), (2, 8, 8, 3, 3, 8),
    (3, 1160, 712, 60, 4, 0), (8, 264, 136, 101, 8, 136), (9, 520, 72, 33, 5, 0), (16, 1024, 512, 16, 2, 512),
    (17, 72, 1032, 40, 7, 72), (32, 512, 256, 64, 6, 512), (33, 136, 264, 8, 8, 0), (64, 256, 128, 160, 8, 256),
    (64, 1024, 264, 16, 16, 0), (5, 4096, 64, 256, 8, 0), (1, 7168, 256, 256, 8, 256), (50, 200, 88, 1024, 20, 0),
])
def test_against_64_bits(T, H, I, E, k, Is):
    _run(T, H, I, E, k, Is)


def test_activation_clamp():
    _run(7, 256, 128, 8, 2, 128, c=0.5)


def test_ties_take_the_lower_id():
    router, W1, W2, _, _ = _weights(128, 64, 40)
    router = router[:, :1].expand(-1, 40).contiguous()  # every expert the same logit
    _, idx, w = DecodeLayer(router, W1, W2, 5)(_x(6, 128), return_routing=True)
    assert (idx == torch.arange(5, device="cuda")).all() and (w == w[:, :1]).all()
    assert ((w - 0.2).abs() <= 2.0 ** -24).all()


def test_routing_like_the_routers_own():
    """The same logits through moe_router_topk: the same ids, weights within the order of their sums."""
    router, W1, W2, _, _ = _weights(64, 64, 100)
    eye = torch.eye(64, device="cuda", dtype=BF)
    _, idx, w = DecodeLayer(router, W1, W2, 9)(eye, return_routing=True)  # logits: the router's rows, exactly
    s = B.shape_of(64, 64, 64, 100, 9)
    i2, w2 = torch.empty(64, 9, dtype=torch.int32, device="cuda"), torch.empty(64, 9, device="cuda")
    ws = torch.empty(B.moe_workspace_layout(s).route_bytes, dtype=torch.uint8, device="cuda")
    B.moe_router_topk(s, router.float().contiguous(), i2, w2, ws)
    assert torch.equal(idx, i2) and ((w - w2).abs() <= 2.0 ** -20 * w2).all()


def test_bad_logits():
    router, W1, W2, _, _ = _weights(64, 64, 8)
    router[0, 3], router[1, 5], router[2, 1] = float("nan"), float("inf"), float("-inf")
    x = torch.zeros(4, 64, device="cuda", dtype=BF)
    x[0, 0], x[1, 1], x[2, 2] = 1.0, 1.0, 1.0  # 0 inf is NaN: a bad weight is bad for every token
    _, idx, w = DecodeLayer(router, W1, W2, 8)(x, return_routing=True)
    assert idx.sort(1).values.equal(torch.arange(8, device="cuda", dtype=torch.int32).expand(4, -1))
    l = (x.float() @ router.float()).nan_to_num(nan=float("-inf"), posinf=float("inf"), neginf=float("-inf"))
    order = torch.sort(l, dim=1, descending=True, stable=True).indices
    assert torch.equal(idx.long(), order)


@pytest.mark.parametrize("T,k", [(1, 3), (6, 4), (40, 3), (64, 16)])
def test_given_routing(T, k):
    """Dropped slots, ids that repeat (more than one group of an expert's slots), weights of any sign."""
    H, I, E = 136, 72, 20
    _, W1, W2, S1, S2 = _weights(H, I, E, 40)
    x, g = _x(T, H), torch.Generator(device="cuda").manual_seed(5)
    idx = torch.randint(-2, E + 1, (T, k), generator=g, device="cuda", dtype=torch.int32)
    idx[: T // 2] = torch.where(idx[: T // 2] >= 0, 2, idx[: T // 2])  # one expert for half of the tokens
    w = torch.randn(T, k, generator=g, device="cuda")
    for s1, s2 in ((None, None), (S1, S2)):
        y = DecodeLayer(None, W1, W2, k, s1, s2)(x, idx, w)
        _check_layer(y, x, idx, w, W1, W2, s1, s2)
    none = torch.full_like(idx, -1)
    assert not DecodeLayer(None, W1, W2, k)(x, none, w).any()  # no expert at all
    y = DecodeLayer(None, W1, W2, k, S1, S2)(x, none, w)
    _check_layer(y, x, none, w, W1, W2, S1, S2)


def test_wide_ids_outside_the_experts():
    _, W1, W2, _, _ = _weights(64, 64, 8)
    x = _x(4, 64)
    idx = torch.tensor([[1, 2 ** 32 + 1], [-2 ** 32 + 3, 2], [2 ** 40, -2 ** 40], [2 ** 31, 7]], device="cuda")
    w = torch.rand(4, 2, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda") + 0.5
    y = DecodeLayer(None, W1, W2, 2)(x, idx, w)
    want = DecodeLayer(None, W1, W2, 2)(x, torch.tensor([[1, -1], [-1, 2], [-1, -1], [-1, 7]], device="cuda", dtype=torch.int32), w)
    assert torch.equal(y, want) and not y[2].any()


def test_same_as_the_layer_of_training():
    T, H, I, E, k = 48, 256, 128, 8, 3
    router, W1, W2, _, _ = _weights(H, I, E)
    x = _x(T, H)
    y, idx, w = DecodeLayer(router, W1, W2, k)(x, return_routing=True)
    big = moe_layer(x, W1, W2, idx, w, workspace=MoEWorkspace(T, H, I, E, k))
    # both within their own roundings of the same value: a half step each of y, the slots' outputs and weights
    scale = (y.float().abs() + 1).double()
    assert ((y.double() - big.double()).abs() <= 6 * HALF * scale).all()


def test_rows_do_not_mix():
    layer, x, y = _run(12, 256, 128, 16, 4, 64)
    x2 = x.clone()
    x2[5] = float("nan")
    y2 = layer(x2)
    rows = [t for t in range(12) if t != 5]
    assert torch.equal(y2[rows], y[rows]) and y2[5].isnan().all()


def test_overlapping_calls_and_replays():
    layer, x, y = _run(16, 512, 256, 32, 4, 128)
    other = _x(16, 512, 7)
    y_other = layer(other)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(10):
        for s, v in zip(streams, (x, other)):
            with torch.cuda.stream(s):
                outs.append(layer(v))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(o, (y, y_other)[i % 2]) for i, o in enumerate(outs))
    graphs = []
    for v in (x, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, layer(v, return_routing=True)))
    for _ in range(3):
        for (g, (o, _, _)), want in zip(graphs, (y, y_other)):
            o.fill_(9.0)
            g.replay()
            assert torch.equal(o, want)
    for s, (g, (o, _, _)) in zip(streams, graphs):  # both at once
        s.wait_stream(torch.cuda.current_stream())
        o.fill_(9.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1][0], y) and torch.equal(graphs[1][1][0], y_other)


def test_scratch_needs_no_clearing():
    router, W1, W2, S1, S2 = _weights(264, 136, 12, 72)
    x = _x(11, 264)
    s = B.MoeDecodeShape(11, 264, 136, 12, 3, 72, 0.0)
    n = B.moe_decode_workspace(s)
    out = []
    for fill in (0, 255, 127):
        ws = torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda")
        y, idx, w = torch.full((13, 264), 7.0, device="cuda", dtype=BF), torch.empty(11, 3, dtype=torch.int32, device="cuda"), torch.empty(11, 3, device="cuda")
        for _ in range(2):  # and again on what the first call left
            B.moe_decode_forward(s, x, router, W1, W2, S1, S2, idx, w, ws, y)
        assert (y[11:] == 7.0).all() and (ws[n:] == fill).all()
        out.append(y)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


def test_activation_next_to_the_largest():
    """Activations of 1.99997 2^127 are finite in FP32 and round to infinity in bf16; up to
    16 tokens the down projection takes them to 16 significant bits, which hold them."""
    H, I = 64, 64
    x = torch.zeros(2, H, device="cuda", dtype=BF)
    x[:, :2] = 1.0
    W1, W2 = torch.zeros(1, H, 2 * I, device="cuda", dtype=BF), torch.zeros(1, I, H, device="cuda", dtype=BF)
    W1[0, 0, 0], W1[0, 0, I], W1[0, 1, I] = 1.9921875 * 2.0 ** 63, 2.0 ** 64, 2.0 ** 56
    W2[0, 0] = 2.0 ** -100
    x[1, 0], x[1, 1] = 2.0 ** 64, 0.0  # an up projection of 2^128: an infinity stays one
    idx, w = torch.zeros(2, 1, device="cuda", dtype=torch.int32), torch.ones(2, 1, device="cuda")
    y = DecodeLayer(None, W1, W2, 1)(x, idx, w).double()
    want = 1.9921875 * (1 + 2.0 ** -8) * 2.0 ** 27
    # half a step of y, and the second operand's own rounding
    assert ((y[0] - want).abs() <= (HALF + 2.0 ** -15) * want).all()
    assert (y[1] == float("inf")).all()


def test_weights_cannot_be_swapped_under_a_layer():
    router, W1, W2, S1, S2 = _weights(64, 64, 8, 64)
    layer = DecodeLayer(router, W1, W2, 2, S1, S2)
    x = _x(3, 64)
    y = layer(x)
    for n, t in (("router", router), ("W1", W1), ("W2", W2), ("S1", S1), ("S2", S2)):
        assert getattr(layer, n).data_ptr() == t.data_ptr()
        with pytest.raises(AttributeError):
            setattr(layer, n, t.clone())
    W2.mul_(2)  # the weights themselves are the caller's
    assert not torch.equal(layer(x), y)


def test_no_tokens_and_refusals():
    router, W1, W2, S1, S2 = _weights(64, 64, 8, 64)
    layer = DecodeLayer(router, W1, W2, 2, S1, S2)
    y, idx, w = layer(_x(0, 64), return_routing=True)
    assert y.shape == (0, 64) and idx.shape == (0, 2)
    for bad in (lambda: layer(_x(65, 64)), lambda: layer(_x(2, 72)), lambda: layer(_x(2, 64), idx, w),
                lambda: DecodeLayer(router[:, :7], W1, W2, 2), lambda: DecodeLayer(router, W1, W2[:, :32], 2),
                lambda: DecodeLayer(router, W1, W2, 2, S1), lambda: DecodeLayer(router, W1, W2, 2, S1, S2[:8]),
                lambda: DecodeLayer(None, W1, W2, 2)(_x(2, 64))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: layer(_x(2, 64).float()), lambda: layer(_x(2, 64).cpu()), lambda: DecodeLayer(router.float(), W1, W2, 2),
                lambda: DecodeLayer(router, W1.half(), W2, 2)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(B.MoeError):
        DecodeLayer(router, W1, W2, 9)
    out = torch.empty(3, 64, device="cuda", dtype=BF)
    x = _x(6, 64)[::2]  # strided rows
    assert layer(x, out=out) is out and torch.equal(out, layer(x.contiguous()))


def test_overlapping_calls_that_fill_the_gpu():
    """Two calls at once, each with a block for every SM: none waits for a block that is not running."""
    router, W1, W2, S1, S2 = _weights(1024, 512, 64, 512)
    layer = DecodeLayer(router, W1, W2, 8, S1, S2)
    xs = [_x(32, 1024, s) for s in (3, 4, 5)]
    want = [layer(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(layer(x))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 3]) for i, g in enumerate(got))
