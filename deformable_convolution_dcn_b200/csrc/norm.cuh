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

// Two float32 values in a register pair: one instruction for both (add, mul, fma .f32x2). The kernels here are short
// of issue slots before they are short of bytes (8x200x200x128: 246 instructions for eight values, summed and applied,
// without the pairs).
struct F2 {
    unsigned long long r;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v.r) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ F2 f2(float v) { return f2(v, v); }
__device__ __forceinline__ void split(F2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v.r));
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v.r) : "l"(a.r), "l"(b.r));
    return v;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v.r) : "l"(a.r), "l"(b.r));
    return v;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v.r) : "l"(a.r), "l"(b.r), "l"(c.r));
    return v;
}
__device__ __forceinline__ F2 shfl_xor(F2 v, int o) {
    return F2{__shfl_xor_sync(~0u, v.r, o)};
}

// 16 bytes of a map <-> pairs: two of float32, four of bfloat16
__device__ __forceinline__ void unpack(F2 (&v)[2], const uint4& q) {
    v[0] = f2(__uint_as_float(q.x), __uint_as_float(q.y));
    v[1] = f2(__uint_as_float(q.z), __uint_as_float(q.w));
}
__device__ __forceinline__ void unpack(F2 (&v)[4], const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack(const F2 (&v)[2]) {
    float a, b, c, d;
    split(v[0], a, b);
    split(v[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}
__device__ __forceinline__ uint4 pack(const F2 (&v)[4]) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        split(v[i], a, b);
        h[i] = __floats2bfloat162_rn(a, b);
    }
    return *reinterpret_cast<uint4*>(h);
}

// A thread's values of its channels, P pairs, on their way to mean and squares about it: sums about a level that starts
// at the thread's first value and is moved to the mean of all values so far when they have doubled. So at least half of
// the values lie about the level whenever squares about a mean are formed by a difference, which then costs a bit, however
// far the first value lies from the others (a border of zeros before a level of 1000: rstd off by 1e-7, where sums about
// the first value were off by 2.5e-3). group_norm.cu does the same with unpaired values.
template <int P>
struct Running {
    F2 k[P], u[P], d[P];  // minus the level, the sum and the squares' sum about it
    int n;                // values taken, counted by the caller
    __device__ __forceinline__ void start(const uint4& q) {
        unpack(k, q);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            k[i] = k[i] * f2(-1.f);
            u[i] = d[i] = f2(0.f);
        }
    }
    __device__ __forceinline__ void add(const uint4& q) {
        F2 v[P];
        unpack(v, q);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const F2 e = v[i] + k[i];
            u[i] = u[i] + e;
            d[i] = fma(e, e, d[i]);
        }
    }
    // the level moves to the mean of the n values (to 2^-23 of the way)
    __device__ __forceinline__ void level() {
        const F2 inv = f2(n > 0 ? -rcp_fast((float)n) : 0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const F2 m = u[i] * inv;
            d[i] = fma(u[i], m, d[i]);
            k[i] = k[i] + m;
            u[i] = f2(0.f);
        }
    }
};

// Joins a channel's slots, means at p[r * pitch] and squares about them `slots` rows further, of count_of(r) values each
// (`count` in all), into the first: the mean is taken about the first slot's, the squares about the mean.
template <typename F>
__device__ __forceinline__ void join_slots(float* p, int pitch, int slots, float count, F&& count_of) {
    const float first = p[0];
    float e = 0.f, q = 0.f;
#pragma unroll 8
    for (int r = 1; r < slots; ++r) e = fmaf(count_of(r), p[r * pitch] - first, e);
    const float mean = first + e * rcp_fast(count);
#pragma unroll 8
    for (int r = 0; r < slots; ++r) {
        const float f = p[r * pitch] - mean;
        q += fmaf(count_of(r) * f, f, p[(slots + r) * pitch]);
    }
    p[0] = mean;
    p[slots * pitch] = q < 0.f ? 0.f : q;  // a NaN stays one
}

template <int ACT, bool FAST>
__device__ __forceinline__ F2 act_apply(F2 z) {
    if constexpr (ACT == kActNone) return z;
    float a, b;
    if constexpr (ACT == kActSilu && FAST) {
        split(z * f2(-1.4426950408889634f), a, b);
        split(f2(exp2_fast(a), exp2_fast(b)) + f2(1.f), a, b);
        return z * f2(rcp_fast(a), rcp_fast(b));
    }
    split(z, a, b);
    return f2(act_apply<ACT, FAST>(a), act_apply<ACT, FAST>(b));
}

// relu's slope where z is too near its border for float32 to say the sign: the sign of z in float64
static __device__ __noinline__ bool positive64(float x, float mean, float rstd, float ga, float be) {
    return ((double)x - (double)mean) * (double)rstd * (double)ga + (double)be > 0.0;
}
// Below this |z|, z = hat gamma + beta may have the wrong sign: hat gamma is near -beta there, each off by a few of
// 2^-24 of its size. (Without beta the sign is that of x - mean, which is exact.)
__device__ __forceinline__ float near_border(float be) { return 2.5e-5f * fabsf(be); }

// dz of one value. hat = (x - mean) rstd.
template <int ACT, bool FAST>
__device__ __forceinline__ float dz_of(float gy, float x, float hat, float mean, float rstd, float ga, float be) {
    const float z = fmaf(hat, ga, be);
    if constexpr (ACT == kActRelu) {
        bool up = z > 0.f;
        if (fabsf(z) < near_border(be)) up = positive64(x, mean, rstd, ga, be);
        return up ? gy : 0.f;
    }
    return act_grad<ACT, FAST>(gy, z);
}

// What the backward keeps of its channels (P pairs): -mean, rstd, gamma, beta, and the largest near_border.
template <int P>
struct Channels {
    F2 nmean[P], rstd[P], ga[P], be[P];
    float border;
    __device__ __forceinline__ void set_border() {
        border = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float a, b;
            split(be[i], a, b);
            border = fmaxf(border, fmaxf(near_border(a), near_border(b)));
        }
    }
    // dz and hat = (x - mean) rstd of a vector of x and of grad_y
    template <int ACT, bool FAST>
    __device__ __forceinline__ void dz(const F2 (&x)[P], const F2 (&gy)[P], F2 (&dz)[P], F2 (&hat)[P]) const {
        F2 z[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            hat[i] = (x[i] + nmean[i]) * rstd[i];
            z[i] = fma(hat[i], ga[i], be[i]);
        }
        if constexpr (ACT == kActNone) {
#pragma unroll
            for (int i = 0; i < P; ++i) dz[i] = gy[i];
        } else if constexpr (ACT == kActRelu) {
            float least = 1e30f;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float z0, z1, g0, g1;
                split(z[i], z0, z1);
                split(gy[i], g0, g1);
                least = fminf(least, fminf(fabsf(z0), fabsf(z1)));
                dz[i] = f2(z0 > 0.f ? g0 : 0.f, z1 > 0.f ? g1 : 0.f);
            }
            if (least < border)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    float x0, x1, g0, g1, m0, m1, r0, r1, a0, a1, b0, b1;
                    split(x[i], x0, x1);
                    split(gy[i], g0, g1);
                    split(nmean[i], m0, m1);
                    split(rstd[i], r0, r1);
                    split(ga[i], a0, a1);
                    split(be[i], b0, b1);
                    dz[i] = f2(positive64(x0, -m0, r0, a0, b0) ? g0 : 0.f, positive64(x1, -m1, r1, a1, b1) ? g1 : 0.f);
                }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float z0, z1;
                split(z[i], z0, z1);
                dz[i] = gy[i] * f2(act_slope<ACT, FAST>(z0), act_slope<ACT, FAST>(z1));
            }
        }
    }
};

// The backward's sums: pixels of a thread that are added up in one float32 chain. Runs of them are added up in another
// (in one chain of 1481 equal values, float32 16x200x200x512 with a constant grad_y, grad_beta was off by 312 of 2^-24; now
// by 8).
constexpr int kRun = 64;

// A float in the shared memory of the cluster's CTA `rank`, at the address of its own copy.
__device__ __forceinline__ float ld_cluster(uint32_t addr, int rank) {
    float v;
    asm volatile(
        "{\n\t.reg .b32 r;\n\t"
        "mapa.shared::cluster.u32 r, %1, %2;\n\t"
        "ld.shared::cluster.f32 %0, [r];\n\t}"
        : "=f"(v)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

// grad_beta, grad_gamma: a channel's sums over the samples (sums [B][C]), by one thread: up to kFewSamples of them, by the
// last block to join; more take params_kernel.
constexpr int kFewSamples = 32;
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
