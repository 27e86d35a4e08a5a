// Forward of the dense gated feed-forward block for a few tokens (decoding):
//   h = x W1,  a = silu(h_g) h_u      and      y = a W2
// with W1 [H][2][I] and W2 [I][H] as they are (rows along the output).
//
// Bound by DRAM: every weight is read once and used for few products, so what
// counts is that every SM streams.  A tile of 64 output features (gated: 64 gate
// and the same 64 up features) goes to a cluster of up to four blocks that
// split K; the warps of a block split its part in units of 4 KB of weights with
// the x that they meet, fetched by TMA by each warp for itself, kFewSlots - 1
// ahead.  The FP32 sums of warps and blocks are joined in a fixed order through
// shared memory, every block of the cluster finishing a share of them.
//
// mma m16n8k16 with the weights as A (16 features x 16 of K, transposed out of
// the box by ldmatrix) and eight tokens as B; kNt such groups of tokens.
//
// Measured, 8 tokens (the 256-row tiles of the large form; the weights' bytes at
// the copy rate): 7168 x 2048 20.0 us (32.1; 13.0), 2048 x 1408 8.9 us (20.1;
// 2.6), 7168 x 18432 127 us (165; 117), and 16 tokens 21.7, 10.3 and 133 us
// (29.7, 20.5 and 137).
#include "few_rows.cuh"

namespace moe {

// More than eight tokens: sixteen a job, each weight read once for them.  A
// small block's weights stay in the L2, and two jobs of eight have less to start
// (16 tokens, 512 x 256: 5.8 against 7.7 us; 1160 x 712: 7.8 against 9.0; but
// 2048 x 1408: 11.4 against 10.3, 7168 x 2048: 36.2 against 21.7).
static bool few_two(const moe_ffn_shape& s) { return s.T > 8 && (long long)s.H * s.I > (1 << 20); }

// Up to 16 tokens always; up to 128 while the jobs' tiles are not many more
// than the SMs (us, this form | the large one: 512 x 256, 128 tokens 6.2 | 11.3;
// 1160 x 712, 64: 9.7 | 14.4; 2048 x 1408, 32: 12.2 | 20.9, 96: 16.3 | 22.3, but
// 128, 256 tiles: 33.8 | 22.9; 4096 x 2048, 32: 18.3 | 25.8, but 64, 256 tiles:
// 29.1 | 27.6).
bool ffn_few_takes(const moe_ffn_shape& s) {
    const int per = few_two(s) ? 16 : 8, wide = s.H > s.I ? s.H : s.I;
    return s.T <= 16 || (s.T <= 128 && (long long)((s.T + per - 1) / per) * ((wide + 63) / 64) <= 200);
}

int launch_ffn_few(const moe_ffn_shape& s, const FfnPtrs& f, cudaStream_t st) {
    const bool two = few_two(s);
    int rc;
    CUtensorMap w1, w2, x, act;
    if ((rc = abi_map_nd(&w1, f.W1, 2, {s.I, 2, s.H}, {64, 1, 16}, "W1 (gate/up halves)"))) return rc;
    if ((rc = abi_map_2d(&w2, f.W2, 2, s.I, s.H, s.H, 64, 32, "W2"))) return rc;
    if ((rc = abi_map_2d(&x, f.x, 2, s.T, s.H, s.H, 16, two ? 16 : 8, "x"))) return rc;
    if ((rc = abi_map_2d(&act, f.a, 2, s.T, s.I, s.I, 32, two ? 16 : 8, "a"))) return rc;
    const float clamp = s.activation_clamp > 0.0f ? s.activation_clamp : INFINITY;
    const FewArgs up = {s.T, s.H, s.I, 0, 0, clamp, static_cast<__nv_bfloat16*>(f.a), f.h, f.status, {}};
    int e = two ? launch_few<FEW_GATED, 2>(up, w1, x, false, "ffn_few_gate_up", st)
                : launch_few<FEW_GATED, 1>(up, w1, x, false, "ffn_few_gate_up", st);
    if (e) return abi_cuda_fail(e, "gate and up projection launch");
    const FewArgs down = {s.T, s.I, s.H, 0, 0, clamp, static_cast<__nv_bfloat16*>(f.y), nullptr, f.status, {}};
    e = two ? launch_few<FEW_PLAIN, 2>(down, w2, act, true, "ffn_few_down", st)
            : launch_few<FEW_PLAIN, 1>(down, w2, act, true, "ffn_few_down", st);
    return e ? abi_cuda_fail(e, "down projection launch") : MOE_OK;
}

}  // namespace moe
