// What the linear layer does to its product: bias, activation, residual; and the
// activations' slopes for its backward.
//
//   z = x W + b      y = act(z) + r      dz = dy act'(z)
//   silu       z sig(z)              sig (1 + z (1 - sig))
//   gelu       z Phi(z)              Phi + z phi(z)           Phi, phi: of N(0, 1)
//   gelu_tanh  z sig(2 u)            sig + 2 z u' sig (1 - sig)
//              u = sqrt(2 / pi) (z + 0.044715 z^3)   (z (1 + tanh u) / 2)
// All in FP32; the results are rounded once.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe_internal.h"

namespace moe {

// 1 / (1 + e^-v) within a few units of 2^-23.
__device__ __forceinline__ float sigmoid_fast(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }
// P(N(0, 1) <= z).  With x = |z| / sqrt(2) and t = 1 / (1 + x / 2) the tail is
// erfc(x) / 2 = t exp(g(t) - x^2) / 2 (the form of the Chebyshev fit in W. H. Press et al.,
// Numerical Recipes, section 6.2); g is smooth on (0, 1], here a fit of its own of
// degree 9 of ln(erfc(x) e^(x^2) / t) that errs by 8.2e-8, 3.9e-7 evaluated in FP32: a
// relative error, in the far tail too (where x^2's rounding, 2^-24 x^2, joins it).
// A third of erfcf's instructions: 4096 x 2048 x 2816 forward 52 -> 41 us.
__device__ __forceinline__ float normal_below(float z) {
    const float x = 0.70710678f * fabsf(z), t = __fdividef(1.0f, fmaf(0.5f, x, 1.0f));
    float g = 0.17689466f;
    g = fmaf(g, t, -0.85072311f);
    g = fmaf(g, t, 1.54551778f);
    g = fmaf(g, t, -1.19725316f);
    g = fmaf(g, t, 0.31883283f);
    g = fmaf(g, t, -0.20170770f);
    g = fmaf(g, t, 0.10020892f);
    g = fmaf(g, t, 0.37370207f);
    g = fmaf(g, t, 1.00003991f);
    g = fmaf(g, t, -1.26551212f);
    const float tail = 0.5f * t * __expf(fmaf(-x, x, g));
    return z < 0.0f ? tail : 1.0f - tail;
}

__device__ __forceinline__ float act_apply(int act, float z) {
    if (act == MOE_ACT_SILU) return z * sigmoid_fast(z);
    if (act == MOE_ACT_GELU) return z * normal_below(z);
    if (act == MOE_ACT_GELU_TANH) return z * sigmoid_fast(1.5957691f * z * (1.0f + 0.044715f * z * z));
    return z;
}
template <int kAct>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (kAct == MOE_ACT_SILU) {
        const float s = sigmoid_fast(z);
        return s + z * s * (1.0f - s);
    } else if constexpr (kAct == MOE_ACT_GELU) {
        const float e = __expf(-0.5f * z * z);
        return normal_below(z) + (e > 0.0f ? z * (0.39894228f * e) : 0.0f);
    } else if constexpr (kAct == MOE_ACT_GELU_TANH) {
        const float s = sigmoid_fast(1.5957691f * z * (1.0f + 0.044715f * z * z)), q = s * (1.0f - s);
        // far out q is 0 and the polynomial may be infinite
        return q > 0.0f ? s + z * q * (1.5957691f * (1.0f + 0.134145f * z * z)) : s;
    } else {
        return 1.0f;
    }
}

struct LinearEpi {
    int act;             // MOE_ACT_*
    int bias_f32;        // bias: FP32, or bf16
    const void* bias;    // [F] or null
    const __nv_bfloat16* residual;  // [T][F], rows res_stride apart, or null
    long long res_stride;
    float* z;  // [T][F] or null
    __device__ __forceinline__ float bias_at(int f) const {
        if (!bias) return 0.0f;
        return bias_f32 ? __ldg(static_cast<const float*>(bias) + f)
                        : __bfloat162float(static_cast<const __nv_bfloat16*>(bias)[f]);
    }
    // One element from its product.
    __device__ __forceinline__ float finish(float v, size_t row, int f, int F) const {
        v += bias_at(f);
        if (z) z[row * F + f] = v;
        v = act_apply(act, v);
        return residual ? v + __bfloat162float(residual[row * res_stride + f]) : v;
    }
};

}  // namespace moe
