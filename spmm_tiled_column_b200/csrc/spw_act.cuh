// spw_act.cuh -- the activations of the product epilogues and of the gated block, and their
// derivatives, in fp32.
//
// Forms chosen so that the tails keep their relative accuracy in fp32: GELU as
// z erfc(-z / sqrt 2) / 2 (1 + erf cancels for z << 0), its tanh form as
// z sigma(2 c (z + 0.044715 z^3)) with c = sqrt(2 / pi), since (1 + tanh a) / 2 = sigma(2 a).
// __expf's error (2 ulp plus 2^-23 |x| relative) is far below the half step of the fp16
// results (2^-11).  An infinite argument gives what the formula gives (SiLU(-inf) = NaN).
#pragma once

#include "spw_internal.cuh"

namespace spw {

__device__ inline float sigmoid_f32(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float kGeluTanhC = 0.7978845608028654f;    // sqrt(2 / pi)
constexpr float kSqrtHalf = 0.7071067811865476f;     // sqrt(1 / 2)
constexpr float kInvSqrt2Pi = 0.3989422804014327f;   // 1 / sqrt(2 pi)

__device__ inline float act_f32(float z, int act) {
    switch (act) {
        case SPW_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
        case SPW_ACT_SILU: return __fdividef(z, 1.0f + __expf(-z));
        case SPW_ACT_GELU: return 0.5f * z * erfcf(-z * kSqrtHalf);
        case SPW_ACT_GELU_TANH:
            return __fdividef(z, 1.0f + __expf(-2.0f * kGeluTanhC * (z + 0.044715f * z * z * z)));
        default: return z;
    }
}

// act(z) and act'(z).
__device__ inline void act_grad_f32(float z, int act, float& a, float& slope) {
    switch (act) {
        case SPW_ACT_RELU:
            a = z > 0.0f ? z : (z != z ? z : 0.0f);
            slope = z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
            break;
        case SPW_ACT_SILU: {
            const float s = sigmoid_f32(z);
            a = z * s;
            slope = s * (1.0f + z * (1.0f - s));
            break;
        }
        case SPW_ACT_GELU: {
            const float p = 0.5f * erfcf(-z * kSqrtHalf);
            a = z * p;
            slope = p + z * kInvSqrt2Pi * __expf(-0.5f * z * z);
            break;
        }
        case SPW_ACT_GELU_TANH: {
            const float z2 = z * z;
            const float s = sigmoid_f32(2.0f * kGeluTanhC * (z + 0.044715f * z2 * z));
            a = z * s;
            slope = s + z * s * (1.0f - s) * 2.0f * kGeluTanhC * (1.0f + 3.0f * 0.044715f * z2);
            break;
        }
        default:
            a = z;
            slope = 1.0f;
    }
}

inline bool act_ok(int act) { return act >= SPW_ACT_NONE && act <= SPW_ACT_GELU_TANH; }

}  // namespace spw
