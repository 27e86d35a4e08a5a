// The joint's kernels for f16 rows.
#include "residual_norm.cuh"

namespace moe {

int residual_norm_fwd_f16(const moe_residual_norm_shape& s, const ResNormPtrs& f, cudaStream_t st) {
    return residual_norm_fwd<__half>(s, f, st);
}
int residual_norm_bwd_f16(const moe_residual_norm_shape& s, const ResNormPtrs& f, cudaStream_t st) {
    return residual_norm_bwd<__half>(s, f, st);
}

}  // namespace moe
