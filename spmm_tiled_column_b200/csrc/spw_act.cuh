// spw_act.cuh -- the activations of the product epilogues and of the gated block, and their
// derivatives, in fp32.
//
// Forms chosen so that the tails keep their relative accuracy in fp32: GELU as z Phi(z) with the
// lower tail Phi(-|z|) = erfc(|z| / sqrt 2) / 2 as a product (1 + erf cancels for z << 0), its tanh
// form as z sigma(2 c (z + 0.044715 z^3)) with c = sqrt(2 / pi), since (1 + tanh a) / 2 = sigma(2 a).
// __expf's error (2 ulp plus 2^-23 |x| relative) is far below the half step of the fp16
// results (2^-11).  An infinite argument gives what the formula gives (SiLU(-inf) = NaN).
#pragma once

#include "spw_internal.cuh"

namespace spw {

__device__ inline float sigmoid_f32(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float kGeluTanhC = 0.7978845608028654f;    // sqrt(2 / pi)
constexpr float kInvSqrt2Pi = 0.3989422804014327f;   // 1 / sqrt(2 pi)

// Phi(-|z|) = exp(-z^2 / 2) t Q(t), t = 1 / (1 + |z| / 4).  Q is a polynomial of degree 7 fitted to
// erfcx(|z| / sqrt 2) / (2 t) for |z| <= 40 (least squares, reweighted until the largest relative
// error was level at 1.0e-6; 1.3e-6 as evaluated in fp32).  Against erfcf, which is correct to a few
// ulp, it takes a third of the instructions, and 32 of them do not spill: GELU added 8 us to the product
// of 4096^3 with erfcf and adds 3 with this.  e: exp(-z^2 / 2).
__device__ inline float normal_tail(float z, float e) {
    const float t = __fdividef(1.0f, fmaf(0.25f, fabsf(z), 1.0f));
    float q = -0.03789707f;
    q = fmaf(q, t, 0.08042956f);
    q = fmaf(q, t, 0.015526491f);
    q = fmaf(q, t, 0.06649756f);
    q = fmaf(q, t, 0.083211355f);
    q = fmaf(q, t, 0.09265328f);
    q = fmaf(q, t, 0.09984776f);
    q = fmaf(q, t, 0.09973058f);
    return q * t * e;
}
// Phi(z) from its lower tail (NaN stays NaN).
__device__ inline float normal_cdf(float z, float tail) { return z < 0.0f ? tail : 1.0f - tail; }

__device__ inline float act_f32(float z, int act) {
    switch (act) {
        case SPW_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
        case SPW_ACT_SILU: return __fdividef(z, 1.0f + __expf(-z));
        case SPW_ACT_GELU: return z * normal_cdf(z, normal_tail(z, __expf(-0.5f * z * z)));
        case SPW_ACT_GELU_TANH:
            return __fdividef(z, 1.0f + __expf(-2.0f * kGeluTanhC * (z + 0.044715f * z * z * z)));
        default: return z;
    }
}

// Several values: one branch on the activation, not one for each value.  A warp then passes over
// its own activation's code alone; with a branch for each of 32 values the five activations stand
// interleaved, and the gated block's product of one 64 x 64 tile took 10.0 us where the plain one,
// which skips them, took 6.1.
template <int N>
__device__ inline void act_all(float (&v)[N], int act) {
    switch (act) {
        case SPW_ACT_RELU:
#pragma unroll
            for (int j = 0; j < N; j++) v[j] = act_f32(v[j], SPW_ACT_RELU);
            break;
        case SPW_ACT_SILU:
#pragma unroll
            for (int j = 0; j < N; j++) v[j] = act_f32(v[j], SPW_ACT_SILU);
            break;
        case SPW_ACT_GELU:
#pragma unroll
            for (int j = 0; j < N; j++) v[j] = act_f32(v[j], SPW_ACT_GELU);
            break;
        case SPW_ACT_GELU_TANH:
#pragma unroll
            for (int j = 0; j < N; j++) v[j] = act_f32(v[j], SPW_ACT_GELU_TANH);
            break;
        default: break;
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
            const float e = __expf(-0.5f * z * z);
            const float p = normal_cdf(z, normal_tail(z, e));
            a = z * p;
            slope = p + z * kInvSqrt2Pi * e;
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
