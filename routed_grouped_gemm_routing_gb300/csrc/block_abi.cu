// Host side of the entry points around the routed experts (include/moe_layer.h):
// argument checks and launches.  No allocation, no synchronisation, no host
// read of device data.
#include <cmath>

#include "moe_internal.h"

using namespace moe;

namespace {

constexpr int kMaxW4K = 65536;
constexpr int kMaxW4N = 1 << 30;  // tiles' and blocks' rows past the last, in 32 bits
constexpr int kMaxNormH = 1 << 29;  // 2 H columns of sums, and a block's stride past the last, in 32 bits

// Alignment that an element of the type needs, 0 for an unknown type.
int elt_size(int type) { return type == MOE_F32 ? 4 : type == MOE_BF16 || type == MOE_F16 ? 2 : 0; }
bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

int check_norm(int64_t rows, int32_t H, int32_t x_type, int32_t w_type) {
    if (rows < 0 || rows >= (1ll << 31)) return abi_fail(MOE_EINVAL, "rows must be in [0, 2^31)");
    if (H < 1 || H > kMaxNormH) return abi_fail(MOE_EINVAL, "H must be in [1, 2^29]");
    if (!elt_size(x_type)) return abi_fail(MOE_EUNSUPPORTED, "x_type must be MOE_BF16, MOE_F16 or MOE_F32");
    if (w_type != MOE_F32 && w_type != x_type)
        return abi_fail(MOE_EUNSUPPORTED, "w_type must be MOE_F32 or x_type");
    return MOE_OK;
}

int check_group(int32_t group) {
    return group == 32 || group == 64 || group == 128
               ? MOE_OK
               : abi_fail(MOE_EUNSUPPORTED, "group must be 32, 64 or 128");
}
int check_w4(const moe_w4_shape* s) {
    if (!s) return abi_fail(MOE_EINVAL, "shape is NULL");
    if (s->T < 0) return abi_fail(MOE_EINVAL, "T must be >= 0");
    if (s->H <= 0 || s->I <= 0) return abi_fail(MOE_EINVAL, "H and I must be > 0");
    if (s->E < 1 || s->E > kMaxExperts) return abi_fail(MOE_EINVAL, "E must be in [1, 1024]");
    if (s->k < 1 || s->k > s->E) return abi_fail(MOE_EINVAL, "k must be in [1, E]");
    if (s->H % 128 || s->I % 128 || s->H > kMaxW4K || s->I > kMaxW4K)
        return abi_fail(MOE_EUNSUPPORTED, "H and I must be multiples of 128, at most 65536");
    if ((long long)s->T * s->k > 65535) return abi_fail(MOE_EUNSUPPORTED, "T*k must be <= 65535");
    if (!std::isfinite(s->activation_clamp)) return abi_fail(MOE_EINVAL, "activation_clamp must be finite");
    return check_group(s->group);
}
int check_ffn(const moe_ffn_shape* s) {
    if (!s) return abi_fail(MOE_EINVAL, "shape is NULL");
    if (s->T < 0) return abi_fail(MOE_EINVAL, "T must be >= 0");
    if (s->H <= 0 || s->I <= 0) return abi_fail(MOE_EINVAL, "H and I must be > 0");
    if (s->H % 8 || s->I % 8) return abi_fail(MOE_EUNSUPPORTED, "H and I must be multiples of 8");
    if (s->T > (1 << 30) || s->H > (1 << 20) || s->I > (1 << 20))
        return abi_fail(MOE_EUNSUPPORTED, "T must be <= 2^30, H and I <= 2^20");
    if (!std::isfinite(s->activation_clamp)) return abi_fail(MOE_EINVAL, "activation_clamp must be finite");
    return MOE_OK;
}
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

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
    const int e = launch_layer_norm_fwd(x_type, w_type, a, st);
    return e ? abi_cuda_fail(e, "layer norm launch") : MOE_OK;
}

int moe_layer_norm_workspace(int64_t rows, int32_t H, size_t* bytes) {
    if (!bytes) return abi_fail(MOE_EINVAL, "bytes is NULL");
    const int rc = check_norm(rows, H, MOE_F32, MOE_F32);
    if (rc) return rc;
    *bytes = (size_t)ln_bwd_parts(rows) * 2 * (size_t)H * sizeof(float);
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
        !aligned(dbias, we) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(ws, 16))
        return abi_fail(MOE_EUNSUPPORTED, "pointers must be aligned to their elements, ws to 16 bytes");
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
    const int e = launch_layer_norm_bwd(x_type, w_type, a, st);
    return e ? abi_cuda_fail(e, "layer norm backward launch") : MOE_OK;
}

int moe_matvec_w4(int32_t M, int32_t N, int32_t K, int32_t group, const void* x, const uint8_t* W_q,
                  const void* W_sf, void* y, void* stream) {
    if (M < 0 || N < 1 || K < 1) return abi_fail(MOE_EINVAL, "M must be >= 0, N and K > 0");
    if (K % 128 || K > kMaxW4K) return abi_fail(MOE_EUNSUPPORTED, "K must be a multiple of 128, at most 65536");
    if (M > 65535) return abi_fail(MOE_EUNSUPPORTED, "M must be <= 65535");
    if (N > kMaxW4N) return abi_fail(MOE_EUNSUPPORTED, "N must be <= 2^30");
    int rc = check_group(group);
    if (rc) return rc;
    if (M == 0) return MOE_OK;
    if (!x || !W_q || !W_sf || !y) return abi_fail(MOE_EINVAL, "NULL pointer argument");
    const void* ptrs[] = {x, W_q, W_sf, y};
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return abi_fail(MOE_EUNSUPPORTED, "pointers must be 16-byte aligned");
    int sms = 0;
    if ((rc = abi_select_device(W_q, &sms))) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    const int e = launch_matvec_w4(M, N, K, group, x, W_q, W_sf, y, st);
    return e ? abi_cuda_fail(e, "4-bit product launch") : MOE_OK;
}

int moe_w4_workspace(const moe_w4_shape* shape, size_t* bytes) {
    if (!bytes) return abi_fail(MOE_EINVAL, "bytes is NULL");
    const int rc = check_w4(shape);
    if (rc) return rc;
    const size_t slots = (size_t)shape->T * shape->k;
    *bytes = up256(slots * shape->I * 2) + slots * shape->H * 4;
    return MOE_OK;
}

int moe_forward_w4(const moe_w4_shape* shape, const void* x, const uint8_t* W1_q, const void* W1_sf,
                   const uint8_t* W2_q, const void* W2_sf, const int32_t* topk_idx, const float* topk_w, void* ws,
                   void* y, void* stream) {
    int rc = check_w4(shape);
    if (rc) return rc;
    if (!topk_idx && (shape->E != 1 || shape->k != 1))
        return abi_fail(MOE_EINVAL, "without topk_idx E and k must be 1");
    if (shape->T == 0) return MOE_OK;
    if (!x || !W1_q || !W1_sf || !W2_q || !W2_sf || !ws || !y || (topk_idx && !topk_w))
        return abi_fail(MOE_EINVAL, "NULL pointer argument");
    const void* ptrs[] = {x, W1_q, W1_sf, W2_q, W2_sf, ws, y};
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return abi_fail(MOE_EUNSUPPORTED, "pointers must be 16-byte aligned");
    // read element by element: one token's routing may start anywhere in a batch's
    if (!aligned(topk_idx, 4) || !aligned(topk_w, 4))
        return abi_fail(MOE_EUNSUPPORTED, "topk_idx and topk_w must be 4-byte aligned");
    int sms = 0;
    if ((rc = abi_select_device(ws, &sms))) return rc;
    uint8_t* w = static_cast<uint8_t*>(ws);
    const size_t slots = (size_t)shape->T * shape->k;
    const W4Experts a = {shape->T, shape->H, shape->I, shape->E, shape->k, shape->group, x, W1_q, W2_q, W1_sf, W2_sf,
                         topk_idx, topk_w, w, reinterpret_cast<float*>(w + up256(slots * shape->I * 2)), y,
                         shape->activation_clamp > 0.0f ? shape->activation_clamp : INFINITY};
    cudaStream_t st = (cudaStream_t)stream;
    const int e = launch_experts_w4(a, st);
    return e ? abi_cuda_fail(e, "4-bit experts launch") : MOE_OK;
}

int moe_quantize_w4(int32_t E, int32_t K, int32_t N, int32_t group, const void* W, uint8_t* W_q, void* W_sf,
                    void* stream) {
    if (E < 1 || E > kMaxExperts || K < 1 || N < 1) return abi_fail(MOE_EINVAL, "E must be in [1, 1024], K and N > 0");
    if (K % 128 || K > kMaxW4K) return abi_fail(MOE_EUNSUPPORTED, "K must be a multiple of 128, at most 65536");
    if (N > kMaxW4N) return abi_fail(MOE_EUNSUPPORTED, "N must be <= 2^30");
    int rc = check_group(group);
    if (rc) return rc;
    if (!W || !W_q || !W_sf) return abi_fail(MOE_EINVAL, "NULL pointer argument");
    const void* ptrs[] = {W, W_q, W_sf};
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return abi_fail(MOE_EUNSUPPORTED, "pointers must be 16-byte aligned");
    int sms = 0;
    if ((rc = abi_select_device(W, &sms))) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    const int e = launch_quantize_w4(E, K, N, group, W, W_q, W_sf, st);
    return e ? abi_cuda_fail(e, "4-bit quantization launch") : MOE_OK;
}

int moe_ffn_workspace_layout(const moe_ffn_shape* shape, moe_ffn_layout* out) {
    if (!out) return abi_fail(MOE_EINVAL, "out is NULL");
    const int rc = check_ffn(shape);
    if (rc) return rc;
    const size_t T = (size_t)shape->T, I = (size_t)shape->I;
    out->a = 0;
    out->h = up256(T * I * 2);
    out->saved_bytes = out->h + up256(T * 2 * I * 4);
    out->status = 0;
    out->dh = 256;
    out->part = out->dh + up256(T * 2 * I * 2);
    out->ws_bytes = out->part + up256((size_t)(shape->T > 0 ? ffn_part_bytes(*shape) : 0));
    return MOE_OK;
}

int moe_ffn_forward(const moe_ffn_shape* shape, const void* x, const void* W1, const void* W2, int32_t for_backward,
                    void* saved, void* ws, void* y, void* stream) {
    moe_ffn_layout L;
    int rc = moe_ffn_workspace_layout(shape, &L);
    if (rc) return rc;
    if (shape->T == 0) return MOE_OK;
    if (!x || !W1 || !W2 || !saved || !ws || !y) return abi_fail(MOE_EINVAL, "NULL pointer argument");
    const void* ptrs[] = {x, W1, W2, saved, ws, y};
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return abi_fail(MOE_EUNSUPPORTED, "pointers must be 16-byte aligned");
    int sms = 0;
    if ((rc = abi_select_device(ws, &sms))) return rc;
    uint8_t *sv = static_cast<uint8_t*>(saved), *w = static_cast<uint8_t*>(ws);
    FfnPtrs f = {};
    f.x = x;
    f.W1 = W1;
    f.W2 = W2;
    f.a = sv + L.a;
    f.h = for_backward ? reinterpret_cast<float*>(sv + L.h) : nullptr;
    f.part = reinterpret_cast<float*>(w + L.part);
    f.status = reinterpret_cast<int32_t*>(w + L.status);
    f.y = y;
    return ffn_few_takes(*shape) ? launch_ffn_few(*shape, f, (cudaStream_t)stream)
                                 : launch_ffn_forward(*shape, f, (cudaStream_t)stream);
}

int moe_ffn_backward(const moe_ffn_shape* shape, const void* dY, const void* x, const void* W1, const void* W2,
                     const void* saved, void* ws, void* dx, void* dW1, void* dW2, void* stream) {
    moe_ffn_layout L;
    int rc = moe_ffn_workspace_layout(shape, &L);
    if (rc) return rc;
    if (!dW1 || !dW2 || (shape->T > 0 && (!dY || !x || !W1 || !W2 || !saved || !ws || !dx)))
        return abi_fail(MOE_EINVAL, "NULL pointer argument");
    const void* ptrs[] = {dY, x, W1, W2, saved, ws, dx, dW1, dW2};
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return abi_fail(MOE_EUNSUPPORTED, "pointers must be 16-byte aligned");
    int sms = 0;
    if ((rc = abi_select_device(dW1, &sms))) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    if (shape->T == 0) {
        const size_t HI = (size_t)shape->H * shape->I;
        cudaError_t ce = cudaMemsetAsync(dW1, 0, HI * 4, st);
        if (ce == cudaSuccess) ce = cudaMemsetAsync(dW2, 0, HI * 2, st);
        return ce == cudaSuccess ? MOE_OK : abi_cuda_fail((int)ce, "zeroing weight gradients");
    }
    uint8_t *sv = static_cast<uint8_t*>(const_cast<void*>(saved)), *w = static_cast<uint8_t*>(ws);
    FfnPtrs f = {};
    f.x = x;
    f.W1 = W1;
    f.W2 = W2;
    f.dY = dY;
    f.a = sv + L.a;
    f.h = reinterpret_cast<float*>(sv + L.h);
    f.dh = w + L.dh;
    f.part = reinterpret_cast<float*>(w + L.part);
    f.status = reinterpret_cast<int32_t*>(w + L.status);
    f.dx = dx;
    f.dW1 = dW1;
    f.dW2 = dW2;
    return launch_ffn_backward(*shape, f, st);
}

}  // extern "C"
