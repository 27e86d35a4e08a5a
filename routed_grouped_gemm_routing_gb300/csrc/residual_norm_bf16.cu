// The joint's kernels for bf16 rows and the size of the partial sums.
#include "residual_norm.cuh"

namespace moe {

long long residual_norm_part_bytes(const moe_residual_norm_shape& s) {
    if (rn_direct(s.rows, s.H, s.x_type == MOE_F32 ? 4 : 2)) return 0;
    const long long blocks = s.H > kRnMaxH ? rn_long_blocks(s.rows, s.H) : s.rows < 152 ? s.rows : 152;
    return blocks * 4 * s.H * 4;
}

int residual_norm_fwd_bf16(const moe_residual_norm_shape& s, const ResNormPtrs& f, cudaStream_t st) {
    return residual_norm_fwd<__nv_bfloat16>(s, f, st);
}
int residual_norm_bwd_bf16(const moe_residual_norm_shape& s, const ResNormPtrs& f, cudaStream_t st) {
    return residual_norm_bwd<__nv_bfloat16>(s, f, st);
}

}  // namespace moe
