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

template <int ACT>
__device__ __forceinline__ float act_apply(float z) {
    if constexpr (ACT == kActRelu) return z < 0.f ? 0.f : z;  // a NaN stays one
    if constexpr (ACT == kActSilu) return z / (1.f + expf(-z));
    if constexpr (ACT == kActGelu) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    return z;
}

// d act / dz. s is the pre-activation z; for relu its output serves as well
// (both are positive at the same places).
template <int ACT>
__device__ __forceinline__ float act_slope(float s) {
    if constexpr (ACT == kActRelu) return s > 0.f ? 1.f : 0.f;
    if constexpr (ACT == kActSilu) {
        const float g = 1.f / (1.f + expf(-s));
        return g * (1.f + s * (1.f - g));
    }
    if constexpr (ACT == kActGelu)
        return 0.5f * (1.f + erff(s * 0.70710678118654752f)) + s * expf(-0.5f * s * s) * 0.39894228040143268f;
    return 1.f;
}

// grad_z = grad_y * act'(s); relu selects, so that an infinite grad_y does not become NaN at slope 0
template <int ACT>
__device__ __forceinline__ float act_grad(float gy, float s) {
    if constexpr (ACT == kActNone) return gy;
    if constexpr (ACT == kActRelu) return s > 0.f ? gy : 0.f;
    return gy * act_slope<ACT>(s);
}

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
