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

// exp(x) through the hardware's 2^x: within 2 + floor(1.17 |x|) ulp for the
// fp32 range (CUDA programming guide), far below the bf16 step of the result
// for the |x| < 90 that matter.
// 1 / (1 + exp(-x)); exp(-x) overflows to inf below -88 and the quotient is 0.
__device__ __forceinline__ float sigmoid32(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;

// z (1 + tanh(v)) / 2 = z / (1 + exp(-2 v)): no cancellation for negative z.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == QZ_ACT_RELU) return fmaxf(z, 0.0f);
    if (ACT == QZ_ACT_SILU) return z * sigmoid32(z);
    if (ACT == QZ_ACT_GELU) return z * sigmoid32(kGelu2 * fmaf(kGeluC * z * z, z, z));
    return z;
}

struct ActPair {
    float value, grad;
};

// act(z) and act'(z).  With e = exp(-|v|) neither sigmoid(v) nor 1 - sigmoid(v)
// cancels; SiLU and GELU are both z sigmoid(v), v = z (a + b z^2), v' = a + 3 b z^2.
__device__ __forceinline__ ActPair act_with_grad(int act, float z) {
    ActPair p;
    if (act == QZ_ACT_SILU || act == QZ_ACT_GELU) {
        const float a = act == QZ_ACT_GELU ? kGelu2 : 1.0f, b = act == QZ_ACT_GELU ? kGelu2 * kGeluC : 0.0f;
        const float z2 = z * z;
        const float v = z * fmaf(b, z2, a);
        const float e = __expf(-fabsf(v));
        const float q = __fdividef(1.0f, 1.0f + e);
        const float eq = e * q;
        const float s = v >= 0.0f ? q : eq;
        p.value = z * s;
        p.grad = fmaf(z * (q * eq), fmaf(3.0f * b, z2, a), s);  // sigmoid(v) (1 - sigmoid(v)) = q e q
    } else if (act == QZ_ACT_RELU) {
        p.value = fmaxf(z, 0.0f);
        p.grad = z > 0.0f ? 1.0f : 0.0f;
    } else {
        p.value = z;
        p.grad = 1.0f;
    }
    return p;
}

}  // namespace qz
