// Host side of the entry points around the routed experts (include/moe_layer.h):
// argument checks and launches.  No allocation, no synchronisation, no host
// read of device data.
#include <cmath>

#include "moe_internal.h"

using namespace moe;

namespace {

// Alignment that an element of the type needs, 0 for an unknown type.
int elt_size(int type) { return type == MOE_F32 ? 4 : type == MOE_BF16 || type == MOE_F16 ? 2 : 0; }
bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

int check_norm(int64_t rows, int32_t H, int32_t x_type, int32_t w_type) {
    if (rows < 0 || rows >= (1ll << 31)) return abi_fail(MOE_EINVAL, "rows must be in [0, 2^31)");
    if (H < 1) return abi_fail(MOE_EINVAL, "H must be >= 1");
    if (!elt_size(x_type)) return abi_fail(MOE_EUNSUPPORTED, "x_type must be MOE_BF16, MOE_F16 or MOE_F32");
    if (w_type != MOE_F32 && w_type != x_type)
        return abi_fail(MOE_EUNSUPPORTED, "w_type must be MOE_F32 or x_type");
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_layer_norm_forward(int64_t rows, int32_t H, int32_t x_type, int32_t w_type, const void* x, int64_t x_stride,
                           const void* weight, const void* bias, float eps, void* y, float* mean, float* rstd,
                           void* stream) {
    int rc = check_norm(rows, H, x_type, w_type);
    if (rc) return rc;
    if (!std::isfinite(eps) || eps < 0.0f) return abi_fail(MOE_EINVAL, "eps must be finite and >= 0");
    if (rows == 0) return MOE_OK;
    if (!x || !weight || !y || !mean || !rstd) return abi_fail(MOE_EINVAL, "NULL pointer argument");
    if (x_stride < H) return abi_fail(MOE_EINVAL, "x_stride must be >= H");
    const int xe = elt_size(x_type), we = elt_size(w_type);
    if (!aligned(x, xe) || !aligned(y, xe) || !aligned(weight, we) || !aligned(bias, we) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return abi_fail(MOE_EUNSUPPORTED, "pointers must be aligned to their elements");
    int sms = 0;
    if ((rc = abi_select_device(x, &sms))) return rc;
    const LnFwdArgs a = {rows, H, x, weight, bias, x_stride, eps, y, mean, rstd};
    cudaStream_t st = (cudaStream_t)stream;
    trace_pre(st);
    const int e = launch_layer_norm_fwd(x_type, w_type, a, st);
    trace_post(st, "layer_norm_fwd");
    return e ? abi_cuda_fail(e, "layer norm launch") : MOE_OK;
}

int moe_layer_norm_workspace(int64_t rows, int32_t H, size_t* bytes) {
    if (!bytes) return abi_fail(MOE_EINVAL, "bytes is NULL");
    const int rc = check_norm(rows, H, MOE_F32, MOE_F32);
    if (rc) return rc;
    *bytes = (size_t)(rows < kLnBwdBlocks ? rows : kLnBwdBlocks) * 2 * (size_t)H * sizeof(float);
    return MOE_OK;
}

int moe_layer_norm_backward(int64_t rows, int32_t H, int32_t x_type, int32_t w_type, const void* dy,
                            int64_t dy_stride, const void* x, int64_t x_stride, const void* weight,
                            const float* mean, const float* rstd, void* dx, void* dweight, void* dbias, void* ws,
                            void* stream) {
    int rc = check_norm(rows, H, x_type, w_type);
    if (rc) return rc;
    if (!dweight || (rows > 0 && (!dy || !x || !weight || !mean || !rstd || !dx || !ws)))
        return abi_fail(MOE_EINVAL, "NULL pointer argument");
    if (rows > 0 && (x_stride < H || dy_stride < H)) return abi_fail(MOE_EINVAL, "strides must be >= H");
    const int xe = elt_size(x_type), we = elt_size(w_type);
    if (!aligned(x, xe) || !aligned(dy, xe) || !aligned(dx, xe) || !aligned(weight, we) || !aligned(dweight, we) ||
        !aligned(dbias, we) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(ws, 4))
        return abi_fail(MOE_EUNSUPPORTED, "pointers must be aligned to their elements");
    int sms = 0;
    if ((rc = abi_select_device(dweight, &sms))) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    if (rows == 0) {
        cudaError_t ce = cudaMemsetAsync(dweight, 0, (size_t)H * we, st);
        if (ce == cudaSuccess && dbias) ce = cudaMemsetAsync(dbias, 0, (size_t)H * we, st);
        return ce == cudaSuccess ? MOE_OK : abi_cuda_fail((int)ce, "zeroing the norm's gradients");
    }
    const LnBwdArgs a = {rows, H, dy, x, weight, dy_stride, x_stride, mean, rstd, dx, dweight, dbias,
                         static_cast<float*>(ws)};
    trace_pre(st);
    const int e = launch_layer_norm_bwd(x_type, w_type, a, st);
    trace_post(st, "layer_norm_bwd");
    return e ? abi_cuda_fail(e, "layer norm backward launch") : MOE_OK;
}

}  // extern "C"
