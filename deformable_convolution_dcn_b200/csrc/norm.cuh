// What the two group normalisation files share: 16-byte vectors, and dz.
#pragma once

#include "act.cuh"
#include "kernels.h"

namespace dcn {

__device__ __forceinline__ void unpack(float (&v)[4], const uint4& q) {
    v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void unpack(float (&v)[8], const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <typename T, int V>
__device__ __forceinline__ uint4 pack(const float (&v)[V]) {
    if constexpr (V == 4) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    } else {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        return *reinterpret_cast<uint4*>(h);
    }
}

// relu's slope where z is too near its border for float32 to say the sign: the sign of z in float64
static __device__ __noinline__ bool positive64(float x, float mean, float rstd, float ga, float be) {
    return ((double)x - (double)mean) * (double)rstd * (double)ga + (double)be > 0.0;
}

// dz of one value. hat = (x - mean) rstd.
template <int ACT, bool FAST>
__device__ __forceinline__ float dz_of(float gy, float x, float hat, float mean, float rstd, float ga, float be) {
    const float z = fmaf(hat, ga, be);
    if constexpr (ACT == kActRelu) {
        bool up = z > 0.f;
        if (fabsf(z) < 1e-5f * (fabsf(hat * ga) + fabsf(be)))
            up = positive64(x, mean, rstd, ga, be);
        return up ? gy : 0.f;
    }
    return act_grad<ACT, FAST>(gy, z);
}

// grad_beta, grad_gamma: a channel's sums over the samples (sums [B][C])
__device__ __forceinline__ void params_of(const NormShape& s, const float2* sums, int c, float* gg, float* gb) {
    float2 v = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int b = 0; b < s.B; ++b) {
        const float2 q = __ldcg(sums + (size_t)b * s.C + c);
        v.x += q.x;
        v.y += q.y;
    }
    if (gb) gb[c] = v.x;
    if (gg) gg[c] = v.y;
}

}  // namespace dcn
