// Activation clamp of the block operators (dense gated feed-forward, 4-bit
// experts) to [-c, c]; c = INFINITY: none.  A NaN is not clamped: it stays one
// (fminf and fmaxf would return the bound), forward and backward.
#pragma once

#include <cuda_runtime.h>

namespace moe {

__device__ __forceinline__ float clamp_keep_nan(float z, float c) {
    float r;
    asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, %2;\n\tmin.NaN.f32 %0, t, %3;\n\t}" : "=f"(r) : "f"(z), "f"(-c), "f"(c));
    return r;
}
// Whether the gradient passes: -c <= z <= c, or z is NaN.
__device__ __forceinline__ float clamp_passes(float z, float c) { return fabsf(z) > c ? 0.0f : 1.0f; }

}  // namespace moe
