// Arithmetic shared by the kernels that rotate Q and K (rope_kv.cu, kv_quant.cu).
#pragma once

#include "common.cuh"

namespace sra {
namespace rope {

// a * b - c * d, accurate to a few ulps of the result (W. Kahan).
__device__ __forceinline__ float diff_of_products(float a, float b, float c, float d) {
    const float w = c * d;
    const float e = fmaf(-c, d, w);  // w - c * d, exactly
    const float f = fmaf(a, b, -w);
    return f + e;
}

// clamp(a x, lo, hi) * g in fp32; a NaN product takes the lower bound (fmaxf
// returns its non-NaN operand), as in the separate UClip kernel.
__device__ __forceinline__ float uclip1(float x, float a, float g, float lo, float hi) {
    return fminf(fmaxf(a * x, lo), hi) * g;
}

}  // namespace rope
}  // namespace sra
