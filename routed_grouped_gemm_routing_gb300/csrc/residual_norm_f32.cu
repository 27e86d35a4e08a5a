// The joint's kernels for FP32 rows.
#include "residual_norm.cuh"

namespace moe {

int residual_norm_fwd_f32(const moe_residual_norm_shape& s, const ResNormPtrs& f, cudaStream_t st) {
    return residual_norm_fwd<float>(s, f, st);
}
int residual_norm_bwd_f32(const moe_residual_norm_shape& s, const ResNormPtrs& f, cudaStream_t st) {
    return residual_norm_bwd<float>(s, f, st);
}

}  // namespace moe
