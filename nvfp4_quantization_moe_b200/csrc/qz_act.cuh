// qz_act.cuh -- activations of the experts' products and their derivatives
// (fp32, sm_100a).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/qz.h"

namespace qz {

// Two fp32 values rounded to nearest-even as a bf16 pair, `lo` in the low half.
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// e^x as 2^(x log2 e) on the special function unit: PTX bounds ex2.approx by 2
// ulp, and the rounded product adds |x| / 2 ulp at most; results below 2^-126
// are 0.  rcp.approx is within 1 ulp.  Both are single instructions, and far
// below the half step of a bf16 result.
__device__ __forceinline__ float fast_exp(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}

__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// max(z, 0) that keeps NaN (fmaxf returns its other operand).
__device__ __forceinline__ float relu(float z) { return z <= 0.0f ? 0.0f : z; }

// 1 / (1 + exp(-x)); exp(-x) overflows to inf below -88 and the quotient is 0.
__device__ __forceinline__ float sigmoid32(float x) { return fast_rcp(1.0f + fast_exp(-x)); }

constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;
// z^2 is taken of at most this |z|, far behind where GELU's sigmoid is 0 or 1: an
// infinite z^2 would make 0 z^2 NaN (SiLU's term of it, GELU's derivative where the
// sigmoid is flat).
constexpr float kActFlat = 1e4f;

struct ActPair {
    float value, grad;
};

// act(z) and act'(z).  With e = exp(-|v|) neither sigmoid(v) nor 1 - sigmoid(v)
// cancels; SiLU and GELU are both z sigmoid(v), v = z (a + b z^2), v' = a + 3 b z^2.
template <int ACT>
__device__ __forceinline__ ActPair act_with_grad(float z) {
    ActPair p;
    if (ACT == QZ_ACT_SILU || ACT == QZ_ACT_GELU) {
        const float w = fminf(fabsf(z), kActFlat), z2 = w * w;
        const float v = ACT == QZ_ACT_GELU ? z * fmaf(kGelu2 * kGeluC, z2, kGelu2) : z;
        const float e = fast_exp(-fabsf(v));
        const float q = fast_rcp(1.0f + e);
        const float eq = e * q;
        const float s = v >= 0.0f ? q : eq;
        const float zr = z * (q * eq);  // z sigmoid(v) (1 - sigmoid(v))
        p.value = z * s;
        p.grad = ACT == QZ_ACT_GELU ? fmaf(zr, fmaf(3.0f * kGelu2 * kGeluC, z2, kGelu2), s) : zr + s;
    } else if (ACT == QZ_ACT_RELU) {
        p.value = relu(z);
        p.grad = z > 0.0f ? 1.0f : 0.0f;
    } else {
        p.value = z;
        p.grad = 1.0f;
    }
    return p;
}

}  // namespace qz
