// The dense gated feed-forward block (a shared expert beside the routed ones),
// forward and backward:
//
//   h = x W1 (gate | up)     a = silu(clamp h_g) clamp h_u     y = a W2
//   da = dY W2^T             dW2 = a^T dY
//   dh_g = da u' sig(g')(1 + g'(1 - sig(g'))) [g passes]
//   dh_u = da silu(g') [u passes]              (g', u': the clamped inputs)
//   dx = dh W1^T             dW1 = x^T dh
//
// Six products of 2 T H I (y, da, dW2) or 4 T H I (h, dx, dW1) operations, all
// bound by the tensor cores from a few hundred tokens on: a step of 8192 x 7168 x
// 2048 takes 1.17 ms in a short burst, 1.85 PFLOP/s, 96 % of the measured bf16
// rate (1.37 ms and 1.58 PFLOP/s, 92 % of the sustained rate, when run for
// seconds under the power limit).  One kernel serves
// them (dense_pair_kernel): D[256 x 256] per pair of SMs, tcgen05 cta_group::2,
// operands by TMA (128-byte swizzle, K blocks of 64) straight from the
// row-major tensors: an operand whose rows run along K is K-major, one whose
// columns are the output's is MN-major, so nothing is ever transposed.  Each
// CTA of the pair loads 128 rows of A and 128 columns of B and holds 128 x 256
// of D in TMEM, twice, so that a tile's epilogue runs under the next one's
// products.  The epilogues do the rest of the block on the accumulators:
//   EPI_GATED  the tile's columns are 128 gate features (the first CTA's B) and
//              the same 128 up features (the second's): both projections, the
//              activation and the product in one kernel.  Leaves a and, for the
//              backward, h.
//   EPI_DGATE  dh from da in TMEM and h by TMA, both halves at once.
//   EPI_PLAIN  bf16 D.
//   EPI_PART   FP32 partial sums of a K range (see below).
//
// Roundings: a and dh are operands of bf16 products and are rounded once each.
// h stays FP32 for the backward: its rounding would come on top of dh's (dx and
// dW1 would err by half as much again), and its bytes, written and read once,
// are a few percent of the block's time.
//
// Few tiles (few tokens): the K range is split over several pairs per tile, each
// leaving FP32 partial sums, and ffn_join adds them in a fixed order and applies
// the epilogue; every SM then streams a part of the weights (dense_shape).
// Deterministic in every form: no atomics.
//
// The kernels of a call follow one another by programmatic launches: each
// starts, sets up its barriers and TMEM where an SM is free, and waits for the
// one before it before it touches any tensor.  dW2, dW1 and dx need nothing of
// each other once dh is there: one launch takes the tiles of all three, the
// deepest products first, so that one last round is ragged instead of three
// (4096 x 2048 x 1408: 164 us a step, 186 in three launches; 777 x 1160 x 712:
// 44 and 56 us).
//
// The forward of few tokens (ffn_few_takes) is ffn_few.cu's.
//
// Roles (10 warps per CTA): 0-7 epilogue (warp w: TMEM lanes 32 (w % 4) .. of
// the CTA's 128 rows, every other group of columns from w / 4 on; with four
// warps the arithmetic of EPI_DGATE took longer than the products of a
// 2048-deep tile: 72 -> 38 us at 4096 x 2048 x 1408), 8 TMA producer, 9 MMA
// issuer (first CTA of the pair).  Every wait is bounded; one that runs out
// sets bit 0 of the status word.
//
// The tile is 256 x 256, or narrower (192, 128 columns) where that wastes less of
// the last round over the pairs (dense_shape).
#include "dense_pair.cuh"

namespace moe {

namespace {

Product fwd1(const moe_ffn_shape& s) { return {s.T, s.I, s.H, true}; }
Product fwd2(const moe_ffn_shape& s) { return {s.T, s.H, s.I, false}; }
Product dgate(const moe_ffn_shape& s) { return {s.T, s.I, s.H, false}; }

}  // namespace

long long ffn_part_bytes(const moe_ffn_shape& s) {
    long long most = 0;
    for (const Product& q : {fwd1(s), fwd2(s), dgate(s)})
        if (q.part_bytes() > most) most = q.part_bytes();
    return most;
}

int launch_ffn_forward(const moe_ffn_shape& s, const FfnPtrs& f, cudaStream_t st) {
    const float clamp = s.activation_clamp > 0.0f ? s.activation_clamp : INFINITY;
    int rc;
    {
        const Product q = fwd1(s);
        DenseArgs a = q.args(clamp, f.status);
        a.save_h = f.h != nullptr;
        DenseMaps m = {};
        if ((rc = map_op(&m.a, f.x, s.T, s.H, 128, "x"))) return rc;
        if ((rc = abi_map_nd(&m.b, f.W1, 2, {s.I, 2, s.H}, {64, 1, 64}, "W1 (gate/up halves)"))) return rc;
        int e;
        if (a.splits > 1) {
            if ((rc = abi_map_nd(&m.c0, f.part, 4, {s.I, 2, s.T, a.splits}, {32, 1, 32, 1}, "partial sums"))) return rc;
            e = launch_dense<KN, EPI_PART_GATED>(a, m, "ffn_gate_up", st, true);
            if (!e) e = launch_join<JOIN_GATED>({f.part, s.T, s.I, a.splits, 2, clamp, f.a, f.h}, st);
        } else {
            a.out = static_cast<__nv_bfloat16*>(f.a);
            if (f.h && (rc = abi_map_nd(&m.c1, f.h, 4, {s.I, 2, s.T}, {32, 1, 32}, "h (store)"))) return rc;
            e = launch_dense<KN, EPI_GATED>(a, m, "ffn_gate_up", st, true);
        }
        if (e) return abi_cuda_fail(e, "gate and up projection launch");
    }
    const Product q = fwd2(s);
    DenseArgs a = q.args(clamp, f.status);
    int e;
    if (a.splits > 1) {
        DenseMaps m = {};
        if ((rc = map_op(&m.a, f.a, s.T, s.I, 128, "a"))) return rc;
        if ((rc = map_op(&m.b, f.W2, s.I, s.H, 64, "W2"))) return rc;
        if ((rc = abi_map_nd(&m.c0, f.part, 4, {s.H, 1, s.T, a.splits}, {32, 1, 32, 1}, "partial sums"))) return rc;
        e = launch_dense<KN, EPI_PART>(a, m, "ffn_down", st);
        if (!e) e = launch_join<JOIN_PLAIN>({f.part, s.T, s.H, a.splits, 1, clamp, f.y, nullptr}, st);
    } else {
        PlainMaps m = {};
        PlainArgs pa = {1, {plain(q, a.width, false, true)}, f.status};
        if ((rc = map_op(&m.m[0], f.a, s.T, s.I, 128, "a"))) return rc;
        if ((rc = map_op(&m.m[1], f.W2, s.I, s.H, 64, "W2"))) return rc;
        if ((rc = map_op(&m.m[2], f.y, s.T, s.H, 32, "y (store)"))) return rc;
        e = launch_plain(pa, m, "ffn_down", st);
    }
    return e ? abi_cuda_fail(e, "down projection launch") : MOE_OK;
}

int launch_ffn_backward(const moe_ffn_shape& s, const FfnPtrs& f, cudaStream_t st) {
    const float clamp = s.activation_clamp > 0.0f ? s.activation_clamp : INFINITY;
    int rc, e;
    {  // da = dY W2^T, and dh from it
        const Product q = dgate(s);
        DenseArgs a = q.args(clamp, f.status);
        DenseMaps m = {};
        if ((rc = map_op(&m.a, f.dY, s.T, s.H, 128, "dY"))) return rc;
        if ((rc = map_op(&m.b, f.W2, s.I, s.H, a.width / 2, "W2 (K-major)"))) return rc;
        if (a.splits > 1) {
            if ((rc = abi_map_nd(&m.c0, f.part, 4, {s.I, 1, s.T, a.splits}, {32, 1, 32, 1}, "partial sums"))) return rc;
            e = launch_dense<KK, EPI_PART>(a, m, "ffn_dgate", st, true);
            if (!e) e = launch_join<JOIN_DGATE>({f.part, s.T, s.I, a.splits, 1, clamp, f.dh, f.h}, st);
        } else {
            a.out = static_cast<__nv_bfloat16*>(f.dh);
            if ((rc = abi_map_nd(&m.c1, f.h, 4, {s.I, 2, s.T}, {32, 1, 32}, "h"))) return rc;
            e = launch_dense<KK, EPI_DGATE>(a, m, "ffn_dgate", st, true);
        }
        if (e) return abi_cuda_fail(e, "dh launch");
    }
    // dW2 = a^T dY, dW1 = x^T dh, dx = dh W1^T: the deepest products first
    struct {
        Product q;
        bool a_mn, b_mn;
        const void *A, *B;
        void* D;
    } job[3] = {{{s.I, s.H, s.T, false, false}, true, true, f.a, f.dY, f.dW2},
                {{s.H, 2 * s.I, s.T, false, false}, true, true, f.x, f.dh, f.dW1},
                {{s.T, s.H, 2 * s.I, false, false}, false, false, f.dh, f.W1, f.dx}};
    if (2 * s.I > s.T) {
        const auto dx = job[2];
        job[2] = job[1];
        job[1] = job[0];
        job[0] = dx;
    }
    const Product qs[3] = {job[0].q, job[1].q, job[2].q};
    const int width = joint_width(qs, 3);
    PlainMaps m = {};
    PlainArgs a = {};
    a.n = 3;
    a.status = f.status;
    for (int i = 0; i < 3; ++i) {
        const auto& j = job[i];
        a.p[i] = plain(j.q, width, j.a_mn, j.b_mn);
        // rows and columns of the stored tensors: K x M or M x K, K x N or N x K
        if ((rc = j.a_mn ? map_op(&m.m[3 * i], j.A, j.q.K, j.q.M, 64, "A (MN-major)")
                         : map_op(&m.m[3 * i], j.A, j.q.M, j.q.K, 128, "A")))
            return rc;
        if ((rc = j.b_mn ? map_op(&m.m[3 * i + 1], j.B, j.q.K, j.q.N, 64, "B (MN-major)")
                         : map_op(&m.m[3 * i + 1], j.B, j.q.N, j.q.K, width / 2, "B")))
            return rc;
        if ((rc = map_op(&m.m[3 * i + 2], j.D, j.q.M, j.q.N, 32, "gradient (store)"))) return rc;
    }
    e = launch_plain(a, m, "ffn_grads", st);
    return e ? abi_cuda_fail(e, "gradient launch") : MOE_OK;
}

}  // namespace moe
