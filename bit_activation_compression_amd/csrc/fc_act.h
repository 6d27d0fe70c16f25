// Activations and their slopes in binary32. exp is v_exp_f32 (2^x, 1 ulp) of a
// rounded product, 1 / x is v_rcp_f32 (1 ulp).
//
// GELU is z * Phi(z). Phi's tail, 0.5 * erfc(u / sqrt 2) for u = |z|, is
// exp(-u^2 / 2) * t * Q(t) with t = 1 / (1 + 0.3 u): Q is this library's own
// least-squares fit of erfcx in t (degree 7, reweighted to an even relative error of
// 1.7e-7 on [0, 14.5]; 6e-7 with binary32 steps), so that small values far out on
// the negative side keep their digits.
#pragma once

#include "fc_device.h"

namespace fc {
namespace {

constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;

__device__ __forceinline__ float exp_of(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504f); }

// p = 1 / (1 + exp(-v)), to its own last digits also where it is small, and q = 1 - p,
// to the last digits of 1: what it is multiplied with is small where it vanishes.
__device__ __forceinline__ void sigmoid_pair(float v, float &p, float &q) {
    p = __builtin_amdgcn_rcpf(1.0f + exp_of(-v));
    q = 1.0f - p;
}

// Phi(z), and exp(-z^2 / 2)
__device__ __forceinline__ float normal_cdf(float z, float &bell) {
    const float u = __builtin_fabsf(z);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, u, 1.0f));
    float q = 0.03542386f;
    q = __builtin_fmaf(q, t, -0.15615894f);
    q = __builtin_fmaf(q, t, 0.20455757f);
    q = __builtin_fmaf(q, t, -0.052034684f);
    q = __builtin_fmaf(q, t, 0.12769209f);
    q = __builtin_fmaf(q, t, 0.10017586f);
    q = __builtin_fmaf(q, t, 0.120712146f);
    q = __builtin_fmaf(q, t, 0.119632006f);
    bell = __builtin_amdgcn_exp2f(u * (u * -0.72134752f));
    const float tail = q * t * bell;
    return z < 0.0f ? tail : 1.0f - tail;
}

// c * (z + 0.044715 z^3), c = 2 sqrt(2 / pi): tanh's form of GELU is z * sigmoid of this
__device__ __forceinline__ float gelu_tanh_argument(float z) {
    return z * __builtin_fmaf(z * z, 1.59576912f * 0.044715f, 1.59576912f);
}

// A negative number is 0, a NaN stays (by its bits: the build takes floats for
// numbers).
__device__ __forceinline__ float relu(float z) {
    const uint32_t b = __builtin_bit_cast(uint32_t, z);
    return b - 0x80000000u <= 0x7F800000u ? 0.0f : z;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == kActRelu) {
        return relu(z);
    } else if constexpr (ACT == kActSilu) {
        float p, q;
        sigmoid_pair(z, p, q);
        return z * p;
    } else if constexpr (ACT == kActGelu) {
        float bell;
        return z * normal_cdf(z, bell);
    } else {
        static_assert(ACT == kActGeluTanh, "an activation");
        float p, q;
        sigmoid_pair(gelu_tanh_argument(z), p, q);
        return z * p;
    }
}

// The activation's value and slope at a finite z.
template <int ACT>
__device__ __forceinline__ void act_both(float z, float &value, float &slope) {
    if constexpr (ACT == kActRelu) {
        value = relu(z);
        slope = z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (ACT == kActSilu) {
        float p, q;
        sigmoid_pair(z, p, q);
        value = z * p;
        slope = __builtin_fmaf(value, q, p);
    } else if constexpr (ACT == kActGelu) {
        float bell;
        const float cdf = normal_cdf(z, bell);
        value = z * cdf;
        slope = __builtin_fmaf(z * bell, 0.39894228f, cdf);
    } else {
        static_assert(ACT == kActGeluTanh, "an activation");
        float p, q;
        sigmoid_pair(gelu_tanh_argument(z), p, q);
        value = z * p;
        slope = __builtin_fmaf(value * q, __builtin_fmaf(z * z, 3.0f * 1.59576912f * 0.044715f, 1.59576912f), p);
    }
}

}  // namespace
}  // namespace fc
