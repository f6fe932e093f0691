// Group normalisation with an activation, channels last, in one pass over HBM
// (the formulas stand in group_norm.cu, which runs what does not fit here).
//
// A thread-block cluster keeps one sample's block of channels (whole groups) in
// the shared memory of its CTAs, each a run of pixels: the map is read once,
// the statistics are taken from shared memory (each CTA's mean first, then the
// squares about it, so that a level far from zero costs no digits), the CTAs
// join theirs through distributed shared memory, and the result is written
// from shared memory. Bytes moved: x once and y once; backward x and grad_y once
// and grad_x once, where two passes over HBM move three and five maps.
//
// A slab is at most 96 KB a CTA where the map allows it, so that two CTAs share
// an SM and one reads while the other computes. Threads keep one 16-byte vector
// of channels and walk the pixels.
//
// Measured (bfloat16, relu): 8x50x50x256 11.3 us, backward 17.7; 1x7x10x256 6.4 us, the latency of its
// loads and joins; larger clusters (16) took longer than the queue of group_norm.cu.
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "kernels.h"
#include "norm.cuh"
#include "tc_ptx.cuh"

namespace dcn {
namespace {

// threads a block: the backward keeps twice the parameters in registers
constexpr int NT_FWD = 512, NT_BWD = 256;
constexpr int MAX_CB = 256;                     // channels a block at most
constexpr uint32_t RED_BYTES = NT_FWD * 8 * 4;     // a block's partial sums
constexpr uint32_t SMALL = 96 * 1024;           // slabs of a CTA

struct ClusterPlan {
    bool ok;
    int cb, nb, cs, rows;  // channels a block, blocks, CTAs a cluster, pixels a CTA
    uint32_t slab;         // bytes of one map's slab
};

// Blocks of whole groups that start and end on a vector, at most MAX_CB channels.
// Wide rows first, fewer CTAs a cluster first, as long as the blocks give every SM
// work; then narrower rows (no less than 64 bytes: rows of 32 bytes cost more than
// a second pass saves, 138 us against 92 us on 8x200x200x128), then clusters of
// eight. Clusters of sixteen are left out: few fit the GPU at a time (8x50x50x256 when
// this kernel was first built: 36 us, with eight 12.4).
ClusterPlan cluster_plan(const NormShape& s, int es, int maps) {
    ClusterPlan p = {};
    const int cg = s.C / s.groups, vec = 16 / es;
    if (s.C % vec) return p;
    int unit = cg;
    while (unit % vec) unit += cg;
    if (unit > MAX_CB || s.C % unit) return p;
    for (const int most : {4, 8})
        for (int bytes = std::max(256, unit * es); bytes >= 64; bytes /= 2) {
            const int cb = std::min({bytes / es / unit * unit, MAX_CB / unit * unit, s.C});
            if (cb < unit) continue;
            const int nb = (s.C + cb - 1) / cb;
            for (int cs = 1; cs <= most; cs *= 2) {
                const int rows = (s.HW + cs - 1) / cs;
                if ((double)rows * cb * es * maps > SMALL) continue;
                const bool fills = (long long)s.B * nb * cs >= 148 || rows < 64;
                if (!fills && cs < most) continue;
                if (!fills && bytes > 64) break;  // narrower blocks give more CTAs
                p.ok = true;
                p.cb = cb;
                p.nb = nb;
                p.cs = cs;
                p.rows = rows;
                p.slab = (uint32_t)rows * cb * es;
                return p;
            }
        }
    return p;
}

// Threads of a block over its slab: vector column cx (of tx), pixels ry, ry + ty, ...
struct Lanes {
    int tx, ty, cx, ry;
    __device__ Lanes(int cb, int V, int nt) {
        tx = cb / V;
        ty = nt / tx;
        cx = threadIdx.x % tx;
        ry = threadIdx.x / tx;
    }
};

// Sums per channel over the block's threads of `a`, to red[slot][cb]; returns the number of slots. Where a warp
// holds whole rows of vectors its lanes add up first.
template <int P, int NT>
__device__ __forceinline__ int spread_sums(F2 (&a)[P], const Lanes& l, int cb, float* red) {
    const bool pow2 = (l.tx & (l.tx - 1)) == 0 && l.tx < 32;
    if (pow2) {
        for (int o = l.tx; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < P; ++i) a[i] = a[i] + shfl_xor(a[i], o);
    }
    const int slot = pow2 ? (int)threadIdx.x / 32 : l.ry;
    if (pow2 ? (int)(threadIdx.x % 32) < l.tx : l.ry < l.ty)
#pragma unroll
        for (int i = 0; i < P; ++i) *reinterpret_cast<F2*>(&red[slot * cb + (l.cx * P + i) * 2]) = a[i];
    return pow2 ? NT / 32 : l.ty;
}

// Sums per group of red[slots][cb] to out[g], a warp a group.
template <int NT>
__device__ __forceinline__ void group_sums(const float* red, int slots, int cb, int cg, int ng, float* out) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int g = warp; g < ng; g += NT / 32) {
        float v = 0.f;
        for (int i = lane; i < slots * cg; i += 32) v += red[(i / cg) * cb + g * cg + i % cg];
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
        if (lane == 0) out[g] = v;
    }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(NT_FWD, 2)
    cluster_forward_kernel(const NormShape s, const ClusterPlan p, const T* __restrict__ x, const T* __restrict__ gamma,
                           const T* __restrict__ beta, T* __restrict__ y, float* __restrict__ stats) {
    constexpr int V = 16 / (int)sizeof(T), P = V / 2, NT = NT_FWD;
    extern __shared__ __align__(16) uint8_t smem[];
    uint4* slab = reinterpret_cast<uint4*>(smem);
    float* red = reinterpret_cast<float*>(smem + p.slab);
    float* lmean = red + RED_BYTES / 4;  // [MAX_CB] this CTA's group means, read by the cluster
    float* lm2 = lmean + MAX_CB;         // and squares about them
    float* gmean = lm2 + MAX_CB;         // the groups' mean and rstd
    float* grstd = gmean + MAX_CB;
    const int rank = blockIdx.x % p.cs, blk = blockIdx.x / p.cs % p.nb, b = blockIdx.x / p.cs / p.nb;
    const int cg = s.C / s.groups, c0 = blk * p.cb, cb = min(p.cb, s.C - c0), ng = cb / cg;
    const int r0 = min(rank * p.rows, s.HW), n = min(p.rows, s.HW - r0);
    const Lanes l(cb, V, NT);
    const bool in = l.ry < l.ty;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const T* xp = x + ((size_t)b * s.HW + r0) * s.C + c0 + l.cx * V;
    F2 a[P] = {};
    if (in) {
        int r = l.ry;
        for (; r + 7 * l.ty < n; r += 8 * l.ty) {
            uint4 q[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) q[k] = ptx::ldg_v4_stream(xp + (size_t)(r + k * l.ty) * s.C);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                slab[(r + k * l.ty) * l.tx + l.cx] = q[k];
                F2 v[P];
                unpack(v, q[k]);
#pragma unroll
                for (int i = 0; i < P; ++i) a[i] = a[i] + v[i];
            }
        }
#pragma unroll 4
        for (; r < n; r += l.ty) {
            const uint4 q = ptx::ldg_v4_stream(xp + (size_t)r * s.C);
            slab[r * l.tx + l.cx] = q;
            F2 v[P];
            unpack(v, q);
#pragma unroll
            for (int i = 0; i < P; ++i) a[i] = a[i] + v[i];
        }
    }
    // gamma and beta on their way while the sums are joined
    F2 ga[P], be[P];
    int g0[P], g1[P];  // the pairs' groups
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (l.cx * P + i) * 2;
        ga[i] = f2(gamma && in ? ld1(gamma + c0 + c) : 1.f, gamma && in ? ld1(gamma + c0 + c + 1) : 1.f);
        be[i] = f2(beta && in ? ld1(beta + c0 + c) : 0.f, beta && in ? ld1(beta + c0 + c + 1) : 0.f);
        g0[i] = c / cg;
        g1[i] = (c + 1) / cg;
    }
    int slots = spread_sums<P, NT>(a, l, cb, red);
    __syncthreads();
    group_sums<NT>(red, slots, cb, cg, ng, lmean);
    __syncthreads();
    const float inv = n > 0 ? 1.f / ((float)n * (float)cg) : 0.f;
    F2 m[P];  // minus the mean
#pragma unroll
    for (int i = 0; i < P; ++i) {
        m[i] = f2(-lmean[g0[i]] * inv, -lmean[g1[i]] * inv);
        a[i] = f2(0.f);
    }
    if (in)
#pragma unroll 4
        for (int r = l.ry; r < n; r += l.ty) {
            F2 v[P];
            unpack(v, slab[r * l.tx + l.cx]);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const F2 d = v[i] + m[i];
                a[i] = fma(d, d, a[i]);
            }
        }
    slots = spread_sums<P, NT>(a, l, cb, red);
    __syncthreads();
    group_sums<NT>(red, slots, cb, cg, ng, lm2);
    // the cluster's runs joined: counts are known, means and squares about them come from each CTA
    if (p.cs > 1) ptx::cluster_sync();
    else __syncthreads();
    for (int g = threadIdx.x; g < ng; g += NT) {
        const uint32_t am = ptx::smem_u32(lmean + g), aq = ptx::smem_u32(lm2 + g);
        const float total = (float)s.HW * (float)cg;
        float sum = 0.f, sq = 0.f;
        float mean, var;
        if (p.cs == 1) {
            mean = lmean[g] / total;
            sq = lm2[g];
        } else {
#pragma unroll 4
            for (int k = 0; k < p.cs; ++k) sum += ld_cluster(am, k);
            mean = sum / total;
#pragma unroll 4
            for (int k = 0; k < p.cs; ++k) {
                const float nk = (float)min(p.rows, s.HW - min(k * p.rows, s.HW)) * (float)cg;
                if (nk > 0.f) {
                    const float d = ld_cluster(am, k) / nk - mean;
                    sq += ld_cluster(aq, k) + nk * d * d;
                }
            }
        }
        var = sq / total;
        const float rstd = rsqrtf(var + s.eps);
        gmean[g] = mean;
        grstd[g] = rstd;
        if (stats && rank == 0) {
            float* st = stats + ((size_t)b * s.groups + c0 / cg + g) * 2;
            st[0] = mean;
            st[1] = rstd;
        }
    }
    __syncthreads();
    // this CTA has read the others' sums: they may leave (waited for at the end)
    if (p.cs > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < P; ++i) {
        m[i] = f2(-gmean[g0[i]], -gmean[g1[i]]);
        ga[i] = ga[i] * f2(grstd[g0[i]], grstd[g1[i]]);
    }
    if (in) {
        T* yp = y + ((size_t)b * s.HW + r0) * s.C + c0 + l.cx * V;
#pragma unroll 4
        for (int r = l.ry; r < n; r += l.ty) {
            F2 v[P];
            unpack(v, slab[r * l.tx + l.cx]);
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = act_apply<ACT, kFast<T>>(fma(v[i] + m[i], ga[i], be[i]));
            *reinterpret_cast<uint4*>(yp + (size_t)r * s.C) = pack(v);
        }
    }
    if (p.cs > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// sums[b][c] = (sum dz, sum dz xh) over the sample; gx where asked for
template <typename T, int ACT>
__global__ void __launch_bounds__(NT_BWD, 2)
    cluster_backward_kernel(const NormShape s, const ClusterPlan p, const T* __restrict__ x, const T* __restrict__ gamma,
                            const T* __restrict__ beta, const float* __restrict__ stats, const T* __restrict__ gy,
                            float2* __restrict__ sums, T* __restrict__ gx) {
    constexpr int V = 16 / (int)sizeof(T), P = V / 2, NT = NT_BWD;
    extern __shared__ __align__(16) uint8_t smem[];
    uint4* slab = reinterpret_cast<uint4*>(smem);
    uint4* slab2 = reinterpret_cast<uint4*>(smem + p.slab);
    float* red = reinterpret_cast<float*>(smem + 2 * p.slab);
    float* lch = red + RED_BYTES / 4;    // [2][MAX_CB] this CTA's sums of a channel, read by the cluster
    float* gc = lch + 2 * MAX_CB;        // [2][MAX_CB] the sample's, times gamma: then c1, c2 of the groups
    const int rank = blockIdx.x % p.cs, blk = blockIdx.x / p.cs % p.nb, b = blockIdx.x / p.cs / p.nb;
    const int cg = s.C / s.groups, c0 = blk * p.cb, cb = min(p.cb, s.C - c0), ng = cb / cg;
    const int r0 = min(rank * p.rows, s.HW), n = min(p.rows, s.HW - r0);
    const Lanes l(cb, V, NT);
    const bool in = l.ry < l.ty;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    Channels<P> ch;
    F2 s1[P] = {}, s2[P] = {};
    int g0[P], g1[P];  // the pairs' groups within the block
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (l.cx * P + i) * 2;
        g0[i] = c / cg;
        g1[i] = (c + 1) / cg;
        const float* st = stats + ((size_t)b * s.groups + c0 / cg) * 2;
        ch.nmean[i] = f2(-__ldg(st + 2 * g0[i]), -__ldg(st + 2 * g1[i]));
        ch.rstd[i] = f2(__ldg(st + 2 * g0[i] + 1), __ldg(st + 2 * g1[i] + 1));
        ch.ga[i] = f2(gamma ? ld1(gamma + c0 + c) : 1.f, gamma ? ld1(gamma + c0 + c + 1) : 1.f);
        ch.be[i] = f2(beta ? ld1(beta + c0 + c) : 0.f, beta ? ld1(beta + c0 + c + 1) : 0.f);
    }
    ch.set_border();
    const size_t at = ((size_t)b * s.HW + r0) * s.C + c0 + l.cx * V;
    auto take = [&](const uint4& qx, const uint4& qg) {
        F2 v[P], g[P], dz[P], hat[P];
        unpack(v, qx);
        unpack(g, qg);
        ch.template dz<ACT, kFast<T>>(v, g, dz, hat);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            s1[i] = s1[i] + dz[i];
            s2[i] = fma(dz[i], hat[i], s2[i]);
        }
    };
    if (in) {
        int r = l.ry;
        for (; r + 3 * l.ty < n; r += 4 * l.ty) {
            uint4 q[4], h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) q[k] = ptx::ldg_v4_stream(x + at + (size_t)(r + k * l.ty) * s.C);
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = ptx::ldg_v4_stream(gy + at + (size_t)(r + k * l.ty) * s.C);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                slab[(r + k * l.ty) * l.tx + l.cx] = q[k];
                slab2[(r + k * l.ty) * l.tx + l.cx] = h[k];
                take(q[k], h[k]);
            }
        }
        for (; r < n; r += l.ty) {
            const uint4 q = ptx::ldg_v4_stream(x + at + (size_t)r * s.C);
            const uint4 h = ptx::ldg_v4_stream(gy + at + (size_t)r * s.C);
            slab[r * l.tx + l.cx] = q;
            slab2[r * l.tx + l.cx] = h;
            take(q, h);
        }
    }
    // sums of a channel over the CTA
    for (int k = 0; k < 2; ++k) {
        const int slots = spread_sums<P, NT>(k ? s2 : s1, l, cb, red);
        __syncthreads();
        for (int c = threadIdx.x; c < cb; c += NT) {
            float v = 0.f;
            for (int i = 0; i < slots; ++i) v += red[i * cb + c];
            lch[k * MAX_CB + c] = v;
        }
        __syncthreads();
    }
    if (p.cs > 1) ptx::cluster_sync();
    for (int i = threadIdx.x; i < 2 * cb; i += NT) {
        const int k = i >= cb, c = i - k * cb;
        const uint32_t addr = ptx::smem_u32(lch + k * MAX_CB + c);
        float v = 0.f;
        if (p.cs == 1) {
            v = lch[k * MAX_CB + c];
        } else {
#pragma unroll 4
            for (int r = 0; r < p.cs; ++r) v += ld_cluster(addr, r);
        }
        if (rank == 0 && sums) reinterpret_cast<float*>(sums + (size_t)b * s.C + c0 + c)[k] = v;
        gc[k * MAX_CB + c] = v * (gamma ? ld1(gamma + c0 + c) : 1.f);
    }
    __syncthreads();
    if (p.cs > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    if (gx) {
        // c1 and c2 of the groups, into red (free by now)
        const float inv = 1.f / ((float)s.HW * (float)cg);
        for (int i = threadIdx.x; i < 2 * ng; i += NT) {
            const int k = i >= ng, g = i - k * ng;
            float v = 0.f;
            for (int c = 0; c < cg; ++c) v += gc[k * MAX_CB + g * cg + c];
            red[k * MAX_CB + g] = v * inv;
        }
        __syncthreads();
        if (in) {
            F2 c1[P], c2[P];  // negated
#pragma unroll
            for (int i = 0; i < P; ++i) {
                c1[i] = f2(-red[g0[i]], -red[g1[i]]);
                c2[i] = f2(-red[MAX_CB + g0[i]], -red[MAX_CB + g1[i]]);
            }
#pragma unroll 2
            for (int r = l.ry; r < n; r += l.ty) {
                F2 v[P], g[P], dz[P], hat[P];
                unpack(v, slab[r * l.tx + l.cx]);
                unpack(g, slab2[r * l.tx + l.cx]);
                ch.template dz<ACT, kFast<T>>(v, g, dz, hat);
#pragma unroll
                for (int i = 0; i < P; ++i) v[i] = ch.rstd[i] * fma(hat[i], c2[i], fma(ch.ga[i], dz[i], c1[i]));
                *reinterpret_cast<uint4*>(gx + at + (size_t)r * s.C) = pack(v);
            }
        }
    }
    if (p.cs > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

template <typename F, typename... Q>
cudaError_t launch(F f, DeviceFlags& flags, const ClusterPlan& p, const NormShape& s, int maps, cudaStream_t st,
                   Q... args) {
    cudaError_t e = max_dynamic_smem_once((const void*)f, SMALL + RED_BYTES + 4 * MAX_CB * 4, flags);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)s.B * p.nb * p.cs));
    cfg.blockDim = dim3(maps == 1 ? NT_FWD : NT_BWD);
    cfg.dynamicSmemBytes = maps * p.slab + RED_BYTES + 4 * MAX_CB * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, f, s, p, args...);
}

template <typename T>
cudaError_t forward_t(const NormShape& s, const ClusterPlan& p, const T* x, const T* gamma, const T* beta, T* y,
                      float* stats, cudaStream_t st) {
    return with_act(s.act, [&](auto A) {
        static DeviceFlags flags;
        return launch(cluster_forward_kernel<T, decltype(A)::value>, flags, p, s, 1, st, x, gamma, beta, y, stats);
    });
}

template <typename T>
cudaError_t backward_t(const NormShape& s, const ClusterPlan& p, const T* x, const T* gamma, const T* beta,
                       const float* stats, const T* gy, float2* sums, T* gx, cudaStream_t st) {
    return with_act(s.act, [&](auto A) {
        static DeviceFlags flags;
        return launch(cluster_backward_kernel<T, decltype(A)::value>, flags, p, s, 2, st, x, gamma, beta, stats, gy, sums,
                      gx);
    });
}

}  // namespace

bool norm_cluster_supported(const NormShape& s, int bf, bool backward) {
    return cluster_plan(s, bf ? 2 : 4, backward ? 2 : 1).ok;
}

cudaError_t norm_cluster_forward(const NormShape& s, int bf, const void* x, const void* gamma, const void* beta,
                                 void* y, float* stats, cudaStream_t st) {
    const ClusterPlan p = cluster_plan(s, bf ? 2 : 4, 1);
    if (!p.ok) return cudaErrorInvalidValue;
    return bf ? forward_t(s, p, (const bf16*)x, (const bf16*)gamma, (const bf16*)beta, (bf16*)y, stats, st)
              : forward_t(s, p, (const float*)x, (const float*)gamma, (const float*)beta, (float*)y, stats, st);
}

cudaError_t norm_cluster_backward(const NormShape& s, int bf, const void* x, const void* gamma, const void* beta,
                                  const float* stats, const void* gy, float2* sums, void* gx, cudaStream_t st) {
    const ClusterPlan p = cluster_plan(s, bf ? 2 : 4, 2);
    if (!p.ok) return cudaErrorInvalidValue;
    return bf ? backward_t(s, p, (const bf16*)x, (const bf16*)gamma, (const bf16*)beta, stats, (const bf16*)gy, sums,
                           (bf16*)gx, st)
              : backward_t(s, p, (const float*)x, (const float*)gamma, (const float*)beta, stats, (const float*)gy,
                           sums, (float*)gx, st);
}

}  // namespace dcn
