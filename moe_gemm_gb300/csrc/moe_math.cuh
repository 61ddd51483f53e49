// SwiGLU in binary32, shared by the kernels of the MoE expert FFN: h must be the same
// number whichever of them makes it.
#pragma once

#include <cuda_runtime.h>

namespace w8a8 {

// e^x in binary32 by Cody and Waite's method: x clamped to [-87, 88], n =
// round-half-even(x log2 e), r = x - n ln2 with ln2 split into a 15-bit head
// (n * head exact) and a tail, e^r by its degree-7 Taylor series (Horner),
// scaled by 2^n. Every step is a separately rounded binary32 operation (the
// _rn intrinsics are never fused into multiply-adds), so the result is a fixed
// function of x, the same in any implementation of these steps.
__device__ __forceinline__ float exp_f32_cw(float x) {
    x = fminf(fmaxf(x, -87.0f), 88.0f);
    const float n = rintf(__fmul_rn(x, 1.44269502163f));
    float r = __fsub_rn(x, __fmul_rn(n, 0.693145751953125f));
    r = __fsub_rn(r, __fmul_rn(n, 1.42860676533018e-06f));
    float p = 1.0f / 5040.0f;
    p = __fadd_rn(__fmul_rn(p, r), 1.0f / 720.0f);
    p = __fadd_rn(__fmul_rn(p, r), 1.0f / 120.0f);
    p = __fadd_rn(__fmul_rn(p, r), 1.0f / 24.0f);
    p = __fadd_rn(__fmul_rn(p, r), 1.0f / 6.0f);
    p = __fadd_rn(__fmul_rn(p, r), 0.5f);
    p = __fadd_rn(__fmul_rn(p, r), 1.0f);
    p = __fadd_rn(__fmul_rn(p, r), 1.0f);
    return __fmul_rn(p, __int_as_float((static_cast<int>(n) + 127) << 23));
}

// h = silu(g) * u = (g / (1 + e^-g)) * u, binary32, IEEE division.
__device__ __forceinline__ float swiglu_f32(float g, float u) {
    const float d = __fadd_rn(1.0f, exp_f32_cw(-g));
    return __fmul_rn(__fdiv_rn(g, d), u);
}

}  // namespace w8a8
