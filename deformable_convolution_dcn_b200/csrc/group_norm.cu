// Group normalisation with an activation, channels last, in two passes over the
// map: for each sample b and group g of C / groups channels, over its
// n = H W C / groups values,
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps),
//   z = gamma (x - mean) rstd + beta,  y = act(z),
// and backward, with xh = (x - mean) rstd and dz = grad_y act'(z),
//   grad_beta = sum_{b,p} dz,  grad_gamma = sum_{b,p} dz xh,
//   c1 = sum_g gamma dz / n,  c2 = sum_g gamma dz xh / n,
//   grad_x = rstd (gamma dz - c1 - xh c2).
//
// The first pass leaves sums of pieces of the map in the workspace, the second
// joins them (in a fixed order) and writes the map. A block covers a run of
// pixels and a block of channels (whole groups where they fit); a thread keeps
// one vector of channels and walks the pixels, so that a warp reads whole
// 128-byte lines and every parameter stays in registers. Sums are float32: the
// statistics are taken about the piece's first pixel and joined as counts,
// means and sums of squares about the mean, so that a level far from zero costs
// no digits.
#include <type_traits>

#include "act.cuh"
#include "kernels.h"
#include "norm.cuh"

namespace dcn {
namespace {

constexpr int NT = 256;         // threads a block
constexpr int MAX_COLS = 1024;  // channels a block at most
constexpr int TARGET = 148 * 4; // blocks that a pass aims at

// How a map is cut. Blocks of cb channels: gpb whole groups, or (gpb = 0) parts
// of one group. chunks runs of rows pixels.
struct Plan {
    int V;       // channels a vector
    int gpb;     // groups a channel block; 0: a group takes `parts` blocks
    int cb;      // channels a block
    int parts;   // blocks a group (gpb = 0), else 1
    int nb;      // channel blocks
    int chunks, rows;
};

Plan make_plan(const NormShape& s, int vec) {
    Plan p = {};
    const int cg = s.C / s.groups;
    p.V = 1;
    if (s.C % vec == 0) {
        // whole groups in blocks that start on a vector
        int unit = 1;
        while ((unit * cg) % vec) ++unit;  // at most vec
        if (unit * cg <= MAX_COLS || s.C <= MAX_COLS) {
            p.V = vec;
            const int u = unit * cg <= MAX_COLS ? MAX_COLS / (unit * cg) * unit : s.groups;
            p.gpb = u < s.groups ? u : s.groups;
        } else if (cg % vec == 0) {
            p.V = vec;
            p.gpb = 0;
        }
    }
    if (p.V == 1) p.gpb = cg <= MAX_COLS / 4 ? (MAX_COLS / 4 / cg < s.groups ? MAX_COLS / 4 / cg : s.groups) : 0;
    if (p.gpb) {
        p.cb = p.gpb * cg;
        p.parts = 1;
        p.nb = (s.groups + p.gpb - 1) / p.gpb;
    } else {
        p.cb = p.V == 1 ? MAX_COLS / 4 : MAX_COLS;
        p.parts = (cg + p.cb - 1) / p.cb;
        p.nb = s.groups * p.parts;
    }
    const int ty = NT / ((p.cb + p.V - 1) / p.V);
    long long want = TARGET / ((long long)s.B * p.nb);
    const long long most = (s.HW + 4LL * ty - 1) / (4LL * ty);  // at least four pixels a thread
    if (want > most) want = most;
    if (want > 128) want = 128;
    if (want < 1) want = 1;
    p.rows = (int)((s.HW + want - 1) / want);
    p.chunks = (int)((s.HW + p.rows - 1) / p.rows);
    return p;
}

// The block's channels [c0, c0 + nc), its groups [g0, g0 + ng), its part of the group.
struct Cols {
    int c0, nc, g0, ng, part;
};
__device__ __forceinline__ Cols cols_of(const NormShape& s, const Plan& p, int blk) {
    const int cg = s.C / s.groups;
    Cols c;
    if (p.gpb) {
        c.g0 = blk * p.gpb;
        c.ng = min(p.gpb, s.groups - c.g0);
        c.c0 = c.g0 * cg;
        c.nc = c.ng * cg;
        c.part = 0;
    } else {
        c.g0 = blk / p.parts;
        c.ng = 1;
        c.part = blk % p.parts;
        c.c0 = c.g0 * cg + c.part * p.cb;
        c.nc = min(p.cb, cg - c.part * p.cb);
    }
    return c;
}

template <typename T, int V>
__device__ __forceinline__ void load(float (&v)[V], const T* p) {
    if constexpr (V == 1)
        v[0] = ld1(p);
    else
        unpack(v, __ldg(reinterpret_cast<const uint4*>(p)));
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&v)[V]) {
    if constexpr (V == 1)
        *p = from_float<T>(v[0]);
    else
        *reinterpret_cast<uint4*>(p) = pack<T>(v);
}

// Joins (n, mean, m2) of two disjoint sets of values.
__device__ __forceinline__ void join(float& n, float& mean, float& m2, float n2, float mean2, float m22) {
    const float t = n + n2;
    if (t == 0.f) return;
    const float d = mean2 - mean, f = n2 / t;
    mean += d * f;
    m2 += m22 + d * d * n * f;
    n = t;
}

// part[((b * chunks + chunk) * groups + g) * parts + part] = (n, mean, m2) of the piece
template <typename T, int V>
__global__ void __launch_bounds__(NT) stats_kernel(const NormShape s, const Plan p, const T* __restrict__ x,
                                                   float4* __restrict__ part) {
    extern __shared__ float sm[];  // [2][ty][cb] sums, reused as [2][cb]
    const Cols c = cols_of(s, p, blockIdx.x % p.nb);
    const int chunk = blockIdx.x / p.nb % p.chunks, b = blockIdx.x / p.nb / p.chunks;
    const int tx = p.cb / V, ty = NT / tx;
    const int cx = threadIdx.x % tx, ry = threadIdx.x / tx;
    const int r0 = chunk * p.rows, r1 = min(r0 + p.rows, s.HW);
    const T* base = x + ((size_t)b * s.HW + r0) * s.C + c.c0 + cx * V;
    float k[V] = {}, s1[V] = {}, s2[V] = {};
    if (cx * V < c.nc && ry < ty) {
        load<T, V>(k, base);
#pragma unroll 4
        for (int r = ry; r < r1 - r0; r += ty) {
            float v[V];
            load<T, V>(v, base + (size_t)r * s.C);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = v[i] - k[i];
                s1[i] += d;
                s2[i] = fmaf(d, d, s2[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sm[ry * p.cb + cx * V + i] = s1[i];
            sm[(ty + ry) * p.cb + cx * V + i] = s2[i];
        }
    }
    __syncthreads();
    const float n = (float)(r1 - r0);
    for (int q = threadIdx.x; q < c.nc; q += NT) {
        float a = 0.f, d = 0.f;
        for (int r = 0; r < ty; ++r) {
            a += sm[r * p.cb + q];
            d += sm[(ty + r) * p.cb + q];
        }
        const float m = a / n;  // about the first pixel
        sm[q] = ld1(x + ((size_t)b * s.HW + r0) * s.C + c.c0 + q) + m;  // row 0's sums were this thread's alone
        const float m2 = d - a * m;
        sm[ty * p.cb + q] = m2 < 0.f ? 0.f : m2;  // a NaN stays one
    }
    __syncthreads();
    // a warp joins a group's channels
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int cw = p.gpb ? s.C / s.groups : c.nc;
    for (int g = warp; g < c.ng; g += NT / 32) {
        float gn = 0.f, gm = 0.f, g2 = 0.f;
        for (int q = lane; q < cw; q += 32) join(gn, gm, g2, n, sm[g * cw + q], sm[ty * p.cb + g * cw + q]);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float n2 = __shfl_down_sync(~0u, gn, o), m2 = __shfl_down_sync(~0u, gm, o),
                        q2 = __shfl_down_sync(~0u, g2, o);
            join(gn, gm, g2, n2, m2, q2);
        }
        if (lane == 0)
            part[(((size_t)b * p.chunks + chunk) * s.groups + c.g0 + g) * p.parts + c.part] =
                make_float4(gn, gm, g2, 0.f);
    }
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(NT) apply_kernel(const NormShape s, const Plan p, const T* __restrict__ x,
                                                   const T* __restrict__ gamma, const T* __restrict__ beta,
                                                   const float4* __restrict__ part, T* __restrict__ y,
                                                   float* __restrict__ stats) {
    extern __shared__ float sm[];  // [2][ng]: mean, rstd
    const Cols c = cols_of(s, p, blockIdx.x % p.nb);
    const int chunk = blockIdx.x / p.nb % p.chunks, b = blockIdx.x / p.nb / p.chunks, cg = s.C / s.groups;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int ngp = p.gpb ? p.gpb : 1;
    for (int g = warp; g < c.ng; g += NT / 32) {
        float n = 0.f, m = 0.f, m2 = 0.f;
        for (int i = lane; i < p.chunks * p.parts; i += 32) {
            const float4 q = part[(((size_t)b * p.chunks + i / p.parts) * s.groups + c.g0 + g) * p.parts + i % p.parts];
            join(n, m, m2, q.x, q.y, q.z);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float n2 = __shfl_down_sync(~0u, n, o), mm = __shfl_down_sync(~0u, m, o),
                        q2 = __shfl_down_sync(~0u, m2, o);
            join(n, m, m2, n2, mm, q2);
        }
        if (lane == 0) {
            const float r = rsqrtf(m2 / ((float)s.HW * (float)cg) + s.eps);
            sm[g] = m;
            sm[ngp + g] = r;
            if (stats && chunk == 0 && c.part == 0) {
                stats[((size_t)b * s.groups + c.g0 + g) * 2] = m;
                stats[((size_t)b * s.groups + c.g0 + g) * 2 + 1] = r;
            }
        }
    }
    __syncthreads();
    const int tx = p.cb / V, ty = NT / tx;
    const int cx = threadIdx.x % tx, ry = threadIdx.x / tx;
    if (cx * V >= c.nc || ry >= ty) return;
    float mean[V], a[V], be[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int ch = cx * V + i, g = p.gpb ? ch / cg : 0;
        mean[i] = sm[g];
        a[i] = sm[ngp + g] * (gamma ? ld1(gamma + c.c0 + ch) : 1.f);
        be[i] = beta ? ld1(beta + c.c0 + ch) : 0.f;
    }
    const int r1 = min((chunk + 1) * p.rows, s.HW);
    const size_t at = (size_t)b * s.HW * s.C + c.c0 + cx * V;
#pragma unroll 4
    for (int r = chunk * p.rows + ry; r < r1; r += ty) {
        float v[V];
        load<T, V>(v, x + at + (size_t)r * s.C);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = act_apply<ACT, kFast<T>>(fmaf(v[i] - mean[i], a[i], be[i]));
        store<T, V>(y + at + (size_t)r * s.C, v);
    }
}

// sums[(b * chunks + chunk) * C + c] = (sum dz, sum dz xh) over the chunk's pixels
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(NT) bwd_sums_kernel(const NormShape s, const Plan p, const T* __restrict__ x,
                                                      const T* __restrict__ gamma, const T* __restrict__ beta,
                                                      const float* __restrict__ stats, const T* __restrict__ gy,
                                                      float2* __restrict__ sums) {
    extern __shared__ float sm[];  // [2][ty][cb]
    const Cols c = cols_of(s, p, blockIdx.x % p.nb);
    const int chunk = blockIdx.x / p.nb % p.chunks, b = blockIdx.x / p.nb / p.chunks, cg = s.C / s.groups;
    const int tx = p.cb / V, ty = NT / tx;
    const int cx = threadIdx.x % tx, ry = threadIdx.x / tx;
    const int r0 = chunk * p.rows, r1 = min(r0 + p.rows, s.HW);
    if (cx * V < c.nc && ry < ty) {
        float mean[V], rstd[V], ga[V], be[V], s1[V] = {}, s2[V] = {};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int ch = c.c0 + cx * V + i;
            const float* st = stats + ((size_t)b * s.groups + ch / cg) * 2;
            mean[i] = __ldg(st);
            rstd[i] = __ldg(st + 1);
            ga[i] = gamma ? ld1(gamma + ch) : 1.f;
            be[i] = beta ? ld1(beta + ch) : 0.f;
        }
        const size_t at = (size_t)b * s.HW * s.C + c.c0 + cx * V;
#pragma unroll 2
        for (int r = r0 + ry; r < r1; r += ty) {
            float v[V], g[V];
            load<T, V>(v, x + at + (size_t)r * s.C);
            load<T, V>(g, gy + at + (size_t)r * s.C);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float hat = (v[i] - mean[i]) * rstd[i];
                const float d = dz_of<ACT, kFast<T>>(g[i], v[i], hat, mean[i], rstd[i], ga[i], be[i]);
                s1[i] += d;
                s2[i] = fmaf(d, hat, s2[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sm[ry * p.cb + cx * V + i] = s1[i];
            sm[(ty + ry) * p.cb + cx * V + i] = s2[i];
        }
    }
    __syncthreads();
    for (int q = threadIdx.x; q < c.nc; q += NT) {
        float a = 0.f, d = 0.f;
        for (int r = 0; r < ty; ++r) {
            a += sm[r * p.cb + q];
            d += sm[(ty + r) * p.cb + q];
        }
        sums[((size_t)b * p.chunks + chunk) * s.C + c.c0 + q] = make_float2(a, d);
    }
}

// grad_beta, grad_gamma: a channel's sums over samples and chunks (32 channels, 8 lanes a block)
__global__ void __launch_bounds__(NT) bwd_params_kernel(const NormShape s, int n, const float2* __restrict__ sums,
                                                        float* __restrict__ ggamma, float* __restrict__ gbeta) {
    __shared__ float2 sm[8][33];
    const int q = threadIdx.x % 32, l = threadIdx.x / 32, c = blockIdx.x * 32 + q;
    float2 t = make_float2(0.f, 0.f);
    if (c < s.C)
        for (int i = l; i < n; i += 8) {
            const float2 v = sums[(size_t)i * s.C + c];
            t.x += v.x;
            t.y += v.y;
        }
    sm[l][q] = t;
    __syncthreads();
    if (l == 0 && c < s.C) {
        for (int i = 1; i < 8; ++i) {
            t.x += sm[i][q].x;
            t.y += sm[i][q].y;
        }
        if (gbeta) gbeta[c] = t.x;
        if (ggamma) ggamma[c] = t.y;
    }
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(NT) bwd_apply_kernel(const NormShape s, const Plan p, const T* __restrict__ x,
                                                       const T* __restrict__ gamma, const T* __restrict__ beta,
                                                       const float* __restrict__ stats, const T* __restrict__ gy,
                                                       const float2* __restrict__ sums, T* __restrict__ gx) {
    extern __shared__ float sm[];  // [2][ng]: c1, c2
    const Cols c = cols_of(s, p, blockIdx.x % p.nb);
    const int chunk = blockIdx.x / p.nb % p.chunks, b = blockIdx.x / p.nb / p.chunks, cg = s.C / s.groups;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int ngp = p.gpb ? p.gpb : 1;
    const float inv = 1.f / ((float)s.HW * (float)cg);
    for (int g = warp; g < c.ng; g += NT / 32) {
        float a = 0.f, d = 0.f;
        for (int i = lane; i < p.chunks * cg; i += 32) {
            const int ch = (c.g0 + g) * cg + i % cg;
            const float2 q = sums[((size_t)b * p.chunks + i / cg) * s.C + ch];
            const float ga = gamma ? ld1(gamma + ch) : 1.f;
            a = fmaf(ga, q.x, a);
            d = fmaf(ga, q.y, d);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            a += __shfl_down_sync(~0u, a, o);
            d += __shfl_down_sync(~0u, d, o);
        }
        if (lane == 0) {
            sm[g] = a * inv;
            sm[ngp + g] = d * inv;
        }
    }
    __syncthreads();
    const int tx = p.cb / V, ty = NT / tx;
    const int cx = threadIdx.x % tx, ry = threadIdx.x / tx;
    if (cx * V >= c.nc || ry >= ty) return;
    float mean[V], rstd[V], ga[V], be[V], c1[V], c2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int ch = c.c0 + cx * V + i, g = p.gpb ? (cx * V + i) / cg : 0;
        const float* st = stats + ((size_t)b * s.groups + ch / cg) * 2;
        mean[i] = __ldg(st);
        rstd[i] = __ldg(st + 1);
        ga[i] = gamma ? ld1(gamma + ch) : 1.f;
        be[i] = beta ? ld1(beta + ch) : 0.f;
        c1[i] = sm[g];
        c2[i] = sm[ngp + g];
    }
    const int r1 = min((chunk + 1) * p.rows, s.HW);
    const size_t at = (size_t)b * s.HW * s.C + c.c0 + cx * V;
#pragma unroll 2
    for (int r = chunk * p.rows + ry; r < r1; r += ty) {
        float v[V], g[V];
        load<T, V>(v, x + at + (size_t)r * s.C);
        load<T, V>(g, gy + at + (size_t)r * s.C);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float hat = (v[i] - mean[i]) * rstd[i];
            const float d = dz_of<ACT, kFast<T>>(g[i], v[i], hat, mean[i], rstd[i], ga[i], be[i]);
            v[i] = rstd[i] * (fmaf(ga[i], d, -c1[i]) - hat * c2[i]);
        }
        store<T, V>(gx + at + (size_t)r * s.C, v);
    }
}

template <typename T>
constexpr int vec_of() {
    return 16 / (int)sizeof(T);
}

int smem_sums(const Plan& p) { return 2 * (NT / (p.cb / p.V)) * p.cb * 4; }
int smem_groups(const Plan& p) { return 2 * (p.gpb ? p.gpb : 1) * 4; }

template <typename T, int V>
cudaError_t forward_v(const NormShape& s, const Plan& p, const T* x, const T* gamma, const T* beta, T* y, float* stats,
                      void* ws, cudaStream_t st, int* launches) {
    const unsigned grid = (unsigned)p.nb * p.chunks * s.B;
    stats_kernel<T, V><<<grid, NT, smem_sums(p), st>>>(s, p, x, (float4*)ws);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
    return with_act(s.act, [&](auto A) {
        apply_kernel<T, V, decltype(A)::value>
            <<<grid, NT, smem_groups(p), st>>>(s, p, x, gamma, beta, (const float4*)ws, y, stats);
        ++*launches;
        return cudaGetLastError();
    });
}

template <typename T, int V>
cudaError_t backward_v(const NormShape& s, const Plan& p, const T* x, const T* gamma, const T* beta,
                       const float* stats, const T* gy, T* gx, float* gg, float* gb, void* ws, cudaStream_t st,
                       int* launches) {
    const unsigned grid = (unsigned)p.nb * p.chunks * s.B;
    return with_act(s.act, [&](auto A) {
        constexpr int ACT = decltype(A)::value;
        bwd_sums_kernel<T, V, ACT><<<grid, NT, smem_sums(p), st>>>(s, p, x, gamma, beta, stats, gy, (float2*)ws);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        ++*launches;
        if (gg || gb) {
            bwd_params_kernel<<<(s.C + 31) / 32, NT, 0, st>>>(s, s.B * p.chunks, (const float2*)ws, gg, gb);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
            ++*launches;
        }
        if (gx) {
            bwd_apply_kernel<T, V, ACT>
                <<<grid, NT, smem_groups(p), st>>>(s, p, x, gamma, beta, stats, gy, (const float2*)ws, gx);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
            ++*launches;
        }
        return e;
    });
}

template <typename T>
cudaError_t forward_t(const NormShape& s, bool vec, const void* x, const void* gamma, const void* beta, void* y,
                      float* stats, void* ws, cudaStream_t st, int* launches) {
    constexpr int V = vec_of<T>();
    const Plan p = make_plan(s, vec ? V : s.C + 1);
    if (p.V == V)
        return forward_v<T, V>(s, p, (const T*)x, (const T*)gamma, (const T*)beta, (T*)y, stats, ws, st, launches);
    return forward_v<T, 1>(s, p, (const T*)x, (const T*)gamma, (const T*)beta, (T*)y, stats, ws, st, launches);
}

template <typename T>
cudaError_t backward_t(const NormShape& s, bool vec, const void* x, const void* gamma, const void* beta,
                       const float* stats, const void* gy, void* gx, float* gg, float* gb, void* ws, cudaStream_t st,
                       int* launches) {
    constexpr int V = vec_of<T>();
    const Plan p = make_plan(s, vec ? V : s.C + 1);
    if (p.V == V)
        return backward_v<T, V>(s, p, (const T*)x, (const T*)gamma, (const T*)beta, stats, (const T*)gy, (T*)gx, gg,
                                gb, ws, st, launches);
    return backward_v<T, 1>(s, p, (const T*)x, (const T*)gamma, (const T*)beta, stats, (const T*)gy, (T*)gx, gg, gb, ws,
                            st, launches);
}

}  // namespace

size_t norm_workspace(const NormShape& s, int bf, bool backward) {
    size_t most = backward ? (size_t)s.B * s.C * sizeof(float2) : 0;  // by clusters
    for (int v : {bf ? 8 : 4, s.C + 1}) {  // vectors, or (an unaligned map) single values
        const Plan p = make_plan(s, v);
        const size_t n = (size_t)s.B * p.chunks;
        const size_t bytes = backward ? n * s.C * sizeof(float2) : n * s.groups * p.parts * sizeof(float4);
        most = bytes > most ? bytes : most;
    }
    return most;
}

cudaError_t norm_forward(const NormShape& s, int bf, bool vec, const void* x, const void* gamma, const void* beta,
                         void* y, float* stats, void* ws, cudaStream_t st, int* launches) {
    if (vec && norm_cluster_supported(s, bf, false)) {
        ++*launches;
        return norm_cluster_forward(s, bf, x, gamma, beta, y, stats, st);
    }
    return bf ? forward_t<bf16>(s, vec, x, gamma, beta, y, stats, ws, st, launches)
              : forward_t<float>(s, vec, x, gamma, beta, y, stats, ws, st, launches);
}

cudaError_t norm_backward(const NormShape& s, int bf, bool vec, const void* x, const void* gamma, const void* beta,
                          const float* stats, const void* gy, void* gx, float* gg, float* gb, void* ws,
                          cudaStream_t st, int* launches) {
    if (vec && norm_cluster_supported(s, bf, true)) {
        float2* sums = gg || gb ? (float2*)ws : nullptr;
        cudaError_t e = norm_cluster_backward(s, bf, x, gamma, beta, stats, gy, sums, gx, st);
        if (e != cudaSuccess) return e;
        ++*launches;
        if (sums) {
            bwd_params_kernel<<<(s.C + 31) / 32, NT, 0, st>>>(s, s.B, (const float2*)ws, gg, gb);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
            ++*launches;
        }
        return e;
    }
    return bf ? backward_t<bf16>(s, vec, x, gamma, beta, stats, gy, gx, gg, gb, ws, st, launches)
              : backward_t<float>(s, vec, x, gamma, beta, stats, gy, gx, gg, gb, ws, st, launches);
}

}  // namespace dcn
