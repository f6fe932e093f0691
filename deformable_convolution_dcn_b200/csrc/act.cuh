// Activations of the linear layer and the group normalisation, and their
// slopes, in float32.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace dcn {

// One element as float32. Loads through a pointer that may be null use this and
// not ldf(): the header's __ldg of a bfloat16 is an inline assembly statement
// that the compiler may move ahead of the test of the pointer, which faults.
__device__ __forceinline__ float ld1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ld1(const bf16* p) {
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}

// dcn_act_t values
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3;

// FAST: the layers of bfloat16 values, forward, where the result is rounded to bfloat16, and backward, where dz goes on to
// float32 sums. Reciprocal and power of two are the hardware's approximations (relative error below 2^-21, results below
// 2^-126 are 0), and the normal distribution's tail is the rational approximation of Abramowitz and Stegun, formula 7.1.26
// (absolute error 1.5e-7 of erf). Backward that is a choice: a slope is off by a few of 2^-22, where the bfloat16 grad_y
// that it multiplies has been rounded at 2^-9; grad_weight of 5000x2048x512 gelu is off by 2.1e-7 by norm (a plain float32
// form, its library product included: 1.3e-6), grad_bias by 1.6e-7 (1.2e-7).
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 1 / (1 + exp(-z))
__device__ __forceinline__ float sigmoid_fast(float z) { return rcp_fast(1.f + exp2_fast(z * -1.4426950408889634f)); }

// e = exp(-z^2 / 2), tail = 1 - Phi(|z|)
__device__ __forceinline__ float normal_tail(float z, float& e) {
    const float t = rcp_fast(fmaf(0.3275911f * 0.70710678118654752f, fabsf(z), 1.f));
    e = exp2_fast(z * z * (-0.5f * 1.4426950408889634f));
    float p = fmaf(0.5f * 1.061405429f, t, 0.5f * -1.453152027f);
    p = fmaf(p, t, 0.5f * 1.421413741f);
    p = fmaf(p, t, 0.5f * -0.284496736f);
    p = fmaf(p, t, 0.5f * 0.254829592f);
    return p * t * e;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act_apply(float z) {
    if constexpr (ACT == kActRelu) {
        float r;
        asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(z));  // a NaN stays one
        return r;
    }
    if constexpr (ACT == kActSilu) return FAST ? z * sigmoid_fast(z) : z / (1.f + expf(-z));
    if constexpr (ACT == kActGelu) {
        if constexpr (FAST) {
            float e;
            const float h = normal_tail(z, e);
            const float zh = h == 0.f ? 0.f : fabsf(z) * h;  // an infinite z times an empty tail is 0
            return fmaxf(z, 0.f) - zh;
        }
        return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    }
    return z;
}

// d act / dz. s is the pre-activation z; for relu its output serves as well
// (both are positive at the same places).
template <int ACT, bool FAST>
__device__ __forceinline__ float act_slope(float s) {
    if constexpr (ACT == kActRelu) return s > 0.f ? 1.f : 0.f;
    if constexpr (ACT == kActSilu) {
        const float g = FAST ? sigmoid_fast(s) : 1.f / (1.f + expf(-s));
        return g * (1.f + s * (1.f - g));
    }
    if constexpr (ACT == kActGelu) {
        if constexpr (FAST) {
            float e;
            const float h = normal_tail(s, e);
            return (s >= 0.f ? 1.f - h : h) + s * e * 0.39894228040143268f;
        }
        return 0.5f * (1.f + erff(s * 0.70710678118654752f)) + s * expf(-0.5f * s * s) * 0.39894228040143268f;
    }
    return 1.f;
}

// grad_z = grad_y * act'(s); relu selects, so that an infinite grad_y does not become NaN at slope 0
template <int ACT, bool FAST>
__device__ __forceinline__ float act_grad(float gy, float s) {
    if constexpr (ACT == kActNone) return gy;
    if constexpr (ACT == kActRelu) return s > 0.f ? gy : 0.f;
    return gy * act_slope<ACT, FAST>(s);
}

// the kernels of a type: bfloat16 takes the fast functions
template <typename T>
constexpr bool kFast = std::is_same<T, bf16>::value;

// Calls f(std::integral_constant<int, ACT>) for the run-time activation.
template <typename F>
inline cudaError_t with_act(int act, F&& f) {
    switch (act) {
        case kActRelu: return f(std::integral_constant<int, kActRelu>{});
        case kActSilu: return f(std::integral_constant<int, kActSilu>{});
        case kActGelu: return f(std::integral_constant<int, kActGelu>{});
        default: return f(std::integral_constant<int, kActNone>{});
    }
}

}  // namespace dcn
