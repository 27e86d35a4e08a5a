"""Products with 4-bit weights against 64 bits.

Tolerance of a product y = sum x (code - 8) sf.  The kernel sums x (128 +
code), exact products of bf16 values, in FP32 from the start value -136 sum x;
every addition of a sum that starts at 136 sum |x| and grows by at most
143 |x| errs by at most 2^-22 of its running size (FP32, truncating adders
allowed), and the additions of a group form chains of at most 16 and the
groups' sums another 2^-24 each: with S = sum_k |x_k| sf_k 280,
|err| <= 16 * 2^-22 * S / 4 = 2^-20 S, and one rounding to bf16, 2^-8 |y|.
The experts: h carries that error into a = silu(g) u (|silu'| <= 1.1), a is
rounded to bf16 (2^-8 |a|), and both go through |W2|."""
import pytest
import torch

from routed_grouped_gemm_routing_gb300 import binding as B
from routed_grouped_gemm_routing_gb300 import build
from routed_grouped_gemm_routing_gb300.block import W4Experts, W4Linear, quantize_w4

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    B.lib()


def _weights(N, K, G, seed, E=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lead = (N,) if E is None else (E, N)
    q = torch.randint(0, 256, (*lead, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sf = ((0.3 + torch.rand((*lead, K // G), generator=g, device="cuda")) / (4.6 * K ** 0.5)).to(BF)
    return q, sf


def _decode(q, sf, G):
    """float64 [N, K], code by code from the format's statement."""
    N, K = q.shape[0], 2 * q.shape[1]
    k = torch.arange(K, device=q.device)
    j, t, i = k % 128 // 32, k % 32 // 8, k % 8
    nib = 8 * (k // 128 * 16 + 4 * t + j) + i // 2 + 4 * (i % 2)
    byte = q[:, nib // 2].int()
    code = torch.where((nib % 2 == 1)[None], byte >> 4, byte & 15)
    return (code - 8).double(), sf.double().repeat_interleave(G, 1)


def _check_product(x, q, sf, G, y):
    c, s = _decode(q, sf, G)
    want = x.double() @ (c * s).t()
    S = 280 * (x.double().abs() @ s.t())
    err = (y.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -20 * S
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("M,N,K,G", [
    (1, 1, 128, 128), (1, 15, 128, 32), (1, 64, 256, 64), (2, 17, 384, 128), (1, 7168, 2048, 128), (7, 1000, 1408, 128),
    (8, 513, 1408, 64), (9, 333, 2048, 32), (12, 1030, 7168, 32), (16, 640, 1024, 64), (17, 48, 2048, 128),
    (33, 200, 7168, 128), (5, 100, 7168, 32), (1, 40, 16384, 64), (8, 32, 14336, 128), (64, 96, 128, 64), (3, 31, 65536, 128),
])
def test_matvec(M, N, K, G):
    q, sf = _weights(N, K, G, M + N)
    x = torch.randn(M, K, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(BF)
    lin = W4Linear(q, sf, G)
    y = lin(x)
    _check_product(x, q, sf, G, y)
    assert torch.equal(y, lin(x))  # fixed order


@pytest.mark.parametrize("M,N,K,G", [(12, 1000, 7168, 128), (16, 333, 7168, 32), (13, 70, 8064, 64), (30, 64, 4224, 128)])
def test_matvec_split_over_k(M, N, K, G):
    """Rows that do not fit one block's shared memory with all of K."""
    q, sf = _weights(N, K, G, M + N)
    x = torch.randn(M, K, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(BF)
    lin = W4Linear(q, sf, G)
    y = lin(x)
    _check_product(x, q, sf, G, y)
    assert torch.equal(y, lin(x))


def test_matvec_last_scale_and_guards():
    """Odd counts of scales (group 128, odd K / 128): nothing past the ends is read into a result or written."""
    N, K, G = 33, 128 * 11, 128
    q, sf = _weights(N, K, G, 5)
    buf = torch.full((N * 11 + 64,), float("nan"), dtype=BF, device="cuda")
    buf[: N * 11] = sf.flatten()
    sf2 = buf[: N * 11].view(N, 11)
    out = torch.full((4 * N + 64,), 7.0, dtype=BF, device="cuda")
    x = torch.randn(4, K, device="cuda").to(BF)
    W4Linear(q, sf2, G).forward(x, out=out[: 4 * N].view(4, N))
    _check_product(x, q, sf, G, out[: 4 * N].view(4, N))
    assert (out[4 * N:] == 7.0).all()


def test_non_finite_rows_stay_in_their_row():
    q, sf = _weights(50, 256, 32, 6)
    x = torch.randn(5, 256, device="cuda").to(BF)
    good = W4Linear(q, sf, 32)(x)
    x2 = x.clone()
    x2[1, 3], x2[3, 200] = float("nan"), float("inf")
    y = W4Linear(q, sf, 32)(x2)
    assert torch.equal(y[[0, 2, 4]], good[[0, 2, 4]]) and y[[1, 3]].isnan().all()


def test_no_rows():
    q, sf = _weights(16, 128, 32, 7)
    assert W4Linear(q, sf, 32)(torch.empty(0, 128, dtype=BF, device="cuda")).shape == (0, 16)


def _experts_ref(x, W1, W2, G, idx, w):
    """(y, tolerance) in 64 bits; W1, W2: (codes, scales)."""
    T, H = x.shape
    y, tol = torch.zeros(T, H, device="cuda", dtype=torch.float64), torch.zeros(T, H, device="cuda", dtype=torch.float64)
    E = W1[0].shape[0]
    xd = x.double()
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if not len(t):
            continue
        c1, s1 = _decode(W1[0][e], W1[1][e], G)
        c2, s2 = _decode(W2[0][e], W2[1][e], G)
        I = c1.shape[0] // 2
        h, dh = xd[t] @ (c1 * s1).t(), 2.0 ** -20 * 280 * (xd[t].abs() @ s1.t())
        g, u = h[:, :I], h[:, I:]
        sg = torch.sigmoid(g)
        a = g * sg * u
        da = 1.1 * dh[:, :I] * u.abs() + (g * sg).abs() * dh[:, I:] + (2.0 ** -8 + 2.0 ** -20) * a.abs()
        ww = w[t, j].double()[:, None]
        y.index_add_(0, t, ww * (a @ (c2 * s2).t()))
        tol.index_add_(0, t, ww.abs() * (da @ (c2 * s2).abs().t() + 2.0 ** -20 * 280 * (a.abs() @ s2.t())))
    return y, tol + 2.0 ** -8 * y.abs()


def _routing(T, E, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w, idx = torch.topk(torch.randn(T, E, generator=g, device="cuda"), k, dim=1)
    return idx.int(), torch.softmax(w, 1)


@pytest.mark.parametrize("T,H,I,E,k,G", [
    (1, 128, 128, 1, 1, 32), (1, 256, 128, 8, 2, 128), (3, 384, 256, 5, 5, 64), (8, 2048, 1408, 16, 6, 128),
    (20, 512, 384, 4, 2, 32), (32, 256, 128, 60, 8, 64), (40, 128, 128, 3, 1, 128), (1, 7168, 2048, 8, 8, 128),
    (9, 7168, 256, 2, 2, 64), (100, 128, 256, 7, 3, 32),
])
def test_experts(T, H, I, E, k, G):
    W1, W2 = _weights(2 * I, H, G, 1, E), _weights(H, I, G, 2, E)
    x = torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(BF)
    idx, w = _routing(T, E, k, 5)
    ex = W4Experts(*W1, *W2, G)
    y = ex(x, idx, w)
    want, tol = _experts_ref(x, W1, W2, G, idx, w)
    err = (y.double() - want).abs()
    assert (err <= tol + 1e-30).all(), float((err / tol.clamp_min(1e-30)).max())
    assert torch.equal(y, ex(x, idx.long(), w.double()))


def test_experts_dropped_slots_and_repeats():
    """Ids outside the experts drop their slot, a token with none gets zeros, one expert may fill several slots."""
    T, H, I, E, k, G = 12, 256, 128, 6, 3, 64
    W1, W2 = _weights(2 * I, H, G, 8, E), _weights(H, I, G, 9, E)
    x = torch.randn(T, H, device="cuda").to(BF)
    idx, w = _routing(T, E, k, 10)
    idx[0] = -1
    idx[1, 1], idx[2, 0], idx[3, 2] = 99, -7, -1
    idx[5] = 2
    idx[6:, 0] = 4
    y = W4Experts(*W1, *W2, G)(x, idx, w)
    want, tol = _experts_ref(x, W1, W2, G, idx, w)
    assert ((y.double() - want).abs() <= tol).all() and not y[0].any()


def test_shared_expert_without_routing():
    H, I, G = 384, 256, 128
    W1, W2 = _weights(2 * I, H, G, 11, 1), _weights(H, I, G, 12, 1)
    for T in (1, 5, 17):
        x = torch.randn(T, H, device="cuda").to(BF)
        y = W4Experts(*W1, *W2, G)(x)
        want, tol = _experts_ref(x, W1, W2, G, torch.zeros(T, 1, dtype=torch.int32, device="cuda"),
                                 torch.ones(T, 1, device="cuda"))
        assert ((y.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("E,K,N,G", [(1, 128, 1, 32), (3, 384, 130, 64), (2, 256, 64, 128)])
def test_quantize(E, K, N, G):
    """Codes and scales follow their definition: exactly, up to a code's tie."""
    W = torch.randn(E, K, N, device="cuda").to(BF)
    W[0, :G, 0] = 0.0
    q, sf = quantize_w4(W, G)
    for e in range(E):
        c, s = _decode(q[e], sf[e], G)
        w = W[e].t().float()
        want = (w.view(N, K // G, G).abs().amax(2) / 7.0).to(BF)
        assert torch.equal(sf[e], want)
        ratio = torch.where(s > 0, w.double() / s.clamp_min(1e-300), torch.zeros_like(s)).clamp(-8, 7)
        assert ((c - ratio).abs() <= 0.5 + 1e-6).all()
        assert ((c * s - w.double()).abs() <= 0.51 * s + 1e-30).all()  # a bf16 scale may fall short of max / 7 by 2^-9


def test_cuda_graph_and_other_stream():
    T, H, I, E, k, G = 4, 256, 128, 8, 2, 32
    W1, W2 = _weights(2 * I, H, G, 13, E), _weights(H, I, G, 14, E)
    x = torch.randn(T, H, device="cuda").to(BF)
    idx, w = _routing(T, E, k, 15)
    ex = W4Experts(*W1, *W2, G)
    want = ex(x, idx, w)
    out = torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ex(x, idx, w, out=out)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        ex(x, idx, w, out=out)
    x.copy_(torch.randn(T, H, device="cuda").to(BF))
    idx.copy_(_routing(T, E, k, 16)[0])
    gr.replay()
    assert torch.equal(out, ex(x, idx, w))


def test_refusals():
    q, sf = _weights(32, 256, 64, 17)
    x = torch.zeros(2, 256, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        W4Linear(q, sf, 48)
    with pytest.raises(ValueError):
        W4Linear(q, sf, 128)
    with pytest.raises(TypeError):
        W4Linear(q.int(), sf, 64)
    lin = W4Linear(q, sf, 64)
    with pytest.raises(ValueError):
        lin(x[:, :128])
    with pytest.raises(TypeError):
        lin(x.float())
    with pytest.raises(ValueError):
        quantize_w4(torch.zeros(100, 8, dtype=BF, device="cuda"), 32)
    with pytest.raises(TypeError):
        quantize_w4(torch.zeros(128, 8, device="cuda"), 32)
    W1, W2 = _weights(256, 256, 64, 18, 2), _weights(256, 128, 64, 19, 2)
    ex = W4Experts(*W1, *W2, 64)
    with pytest.raises(ValueError):
        ex(x)
    with pytest.raises(ValueError):
        ex(x, torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.ones(3, 1, device="cuda"))
    q3, s3 = _weights(32, 192, 64, 20)  # K not a multiple of 128
    with pytest.raises(B.MoeError):
        W4Linear(q3, s3, 64)(torch.zeros(1, 192, dtype=BF, device="cuda"))


@pytest.mark.parametrize("M,N,K,G", [
    (9, 8200, 1152, 32), (12, 16380, 7168, 32), (16, 4100, 2304, 64), (17, 4096, 4096, 128), (32, 3001, 3328, 128),
    (10, 70000, 1024, 128), (16, 1100, 8064, 64), (13, 9000, 1408, 32), (40, 2049, 5120, 64),
])
def test_matvec_sixteen_rows_of_a_large_matrix(M, N, K, G):
    q, sf = _weights(N, K, G, M + N)
    x = torch.randn(M, K, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(BF)
    lin = W4Linear(q, sf, G)
    out = torch.full((M * N + 64,), 7.0, dtype=BF, device="cuda")
    y = lin.forward(x, out=out[: M * N].view(M, N))
    _check_product(x, q, sf, G, y)
    assert torch.equal(y, lin(x)) and (out[M * N:] == 7.0).all()
    x2 = x.clone()
    x2[1, 3], x2[M - 1, K - 1] = float("nan"), float("inf")
    y2 = lin(x2)
    assert torch.equal(y2[2: M - 1], y[2: M - 1]) and torch.equal(y2[0], y[0]) and y2[[1, M - 1]].isnan().all()


@pytest.mark.parametrize("T,H,I,G", [(9, 2048, 2816, 64), (16, 7168, 640, 128), (23, 4096, 2048, 32)])
def test_shared_expert_of_many_rows(T, H, I, G):
    W1, W2 = _weights(2 * I, H, G, 21, 1), _weights(H, I, G, 22, 1)
    x = torch.randn(T, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)).to(BF)
    ex = W4Experts(*W1, *W2, G)
    y = ex(x)
    want, tol = _experts_ref(x, W1, W2, G, torch.zeros(T, 1, dtype=torch.int32, device="cuda"),
                             torch.ones(T, 1, device="cuda"))
    assert ((y.double() - want).abs() <= tol).all() and torch.equal(y, ex(x))
