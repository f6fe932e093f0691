// Group normalisation with an activation, channels last, for long maps of whole
// vectors: the queue of group_norm.cu (units summed first and applied a few sets
// later, from L2) with the loads taken off the threads that compute.
//
// One block an SM. A producer warp claims the units and copies their pixels, which
// lie in one run, to a ring of shared-memory stages (bulk copies, up to 150 KB in
// flight); the other warps compute from there and store. So the memory works on while
// a unit's sums are reduced, joined and released, and those latencies, which bound
// the kernels without the ring (8x200x200x128: 92 us), cost nothing. The producer
// also waits for a set's statistics before it copies a unit of the second pass, and
// leaves them in the unit's first stage.
//
// A claimed unit waits for none but lower ones, which are summed by blocks that
// never wait (see group_norm.cu); the end of a set's sums is looked at before the
// next stage is waited for, so no block's own next unit can hold it up.
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "kernels.h"
#include "norm.cuh"
#include "tc_ptx.cuh"

namespace dcn {
namespace {

// computing threads (and a producer warp): the backward keeps twice the parameters in registers
constexpr int NC_FWD = 768, NC_BWD = 512;
constexpr int MAX_STAGES = 16;
constexpr int MAX_C = 1024;
constexpr int MAX_GROUPS = 256;          // their statistics travel in a stage
constexpr uint32_t RING = 168 * 1024;    // all stages
constexpr uint32_t RED_BYTES = 2 * NC_FWD * 8 * 4;
constexpr long long WAIT_LIMIT = 2000000000LL;

struct StreamPlan {
    bool ok;
    int rows, chunks;      // pixels a unit, units a set (a sample)
    int srows, stages;     // pixels a stage, stages
    uint32_t data, stage;  // bytes of one map's pixels, of a stage
    int lag, grid;
};

StreamPlan stream_plan(const NormShape& s, int es, int maps) {
    StreamPlan p = {};
    const int vec = 16 / es, row = s.C * es;
    if (s.C % vec || s.C > MAX_C || s.groups > MAX_GROUPS) return p;
    const int ty = (maps == 1 ? NC_FWD : NC_BWD) / (s.C / vec);
    // four vectors a thread
    p.srows = std::min(4 / maps * ty, s.HW);
    p.data = (uint32_t)p.srows * row;
    p.stage = maps * p.data + (uint32_t)(s.groups * 8 * maps + 127) / 128 * 128;
    p.stages = (int)std::min<uint32_t>(MAX_STAGES, RING / p.stage);
    // units of 256 KB: their reduction takes about as long as their pixels' way from HBM; smaller ones where the map
    // would not give every SM two
    long long rows = std::max<long long>(1, 256 * 1024 / ((long long)row * maps));
    rows = std::min(rows, std::max<long long>(1, (long long)s.HW * s.B / 296));
    rows = std::max<long long>((rows + p.srows - 1) / p.srows, 1) * p.srows;
    rows = std::max(rows, (s.HW + 255LL) / 256);  // the join walks at most 256 units
    p.rows = (int)std::min<long long>(rows, s.HW);
    p.chunks = (s.HW + p.rows - 1) / p.rows;
    p.lag = (int)std::min<long long>(s.B, 296 / p.chunks + 2);
    p.grid = (int)std::min<long long>(148, (long long)s.B * p.chunks);
    p.ok = true;
    return p;
}

struct Space {
    size_t pieces, sets, total;
};
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
Space space_of(const NormShape& s, const StreamPlan& p, bool backward) {
    Space w;
    w.pieces = up256((2 + 2 * (size_t)s.B) * sizeof(int));  // after the counters
    w.sets = up256(w.pieces + (size_t)s.B * p.chunks * (backward ? s.C : s.groups) * sizeof(float2));
    w.total = up256(w.sets + (size_t)s.B * (backward ? s.C + s.groups : s.groups) * sizeof(float2));
    return w;
}

struct Args {
    NormShape s;
    StreamPlan p;
    int *ticket, *finished, *done, *ready;
    float2 *pieces, *sets;
    unsigned* status;
};

// What the producer says of a stage.
struct Header {
    int pass;   // 0 sums, 1 applies, -1: no more units
    int set, chunk;
    int row0, n;  // its pixels, within the sample
    int first, last;
};

// As in group_norm.cu: unit t of the queue.
__device__ __forceinline__ void unit_at(const Args& a, int t, int& pass, int& set, int& chunk) {
    const int U = a.p.chunks, Q = a.s.B, L = a.p.lag;
    if (t < L * U) {
        pass = 0;
        set = t / U;
        chunk = t % U;
        return;
    }
    int r = t - L * U;
    if (r < (Q - L) * 2 * U) {
        const int i = r / (2 * U), w = r % (2 * U);
        pass = w >= U;
        set = pass ? i : L + i;
        chunk = pass ? w - U : w;
        return;
    }
    r -= (Q - L) * 2 * U;
    pass = 1;
    set = Q - L + r / U;
    chunk = r % U;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

template <int NC>
__device__ __forceinline__ void sync_computing() {
    ptx::bar_sync_named(1, NC);
}

struct Ring {
    uint8_t* smem;
    uint32_t base, full, empty;  // shared addresses: stages, barriers
    Header* headers;
};

// The producer warp. maps: x, or x and grad_y; apply: the second pass is wanted; stats: (mean, rstd) of the backward.
template <typename T, int MAPS>
__device__ __forceinline__ void produce(const Args& a, const Ring& ring, const T* x, const T* gy, const float* stats,
                                        bool apply) {
    const NormShape& s = a.s;
    const StreamPlan& p = a.p;
    const int lane = threadIdx.x % 32;
    const int total = (apply ? 2 : 1) * s.B * p.chunks;
    const uint32_t row = s.C * (uint32_t)sizeof(T);
    int stage = 0;
    uint32_t phase = 1;
    volatile int none = 0;
    bool ok = true;
    int claim = 0;
    if (lane == 0) claim = atomicAdd(a.ticket, 1);
    for (;;) {
        const int t = __shfl_sync(~0u, claim, 0);
        if (t >= total || !ok) break;
        if (lane == 0) claim = atomicAdd(a.ticket, 1);  // the unit after: answered meanwhile
        int pass, set, chunk;
        if (apply) {
            unit_at(a, t, pass, set, chunk);
        } else {
            pass = 0;
            set = t / p.chunks;
            chunk = t % p.chunks;
        }
        if (pass == 1) {  // the set's sums are joined
            const long long t0 = clock64();
            while (ptx::ld_acquire_gpu(a.ready + set) == 0) {
                __nanosleep(100);
                if (clock64() - t0 > WAIT_LIMIT) {
                    atomicOr(a.status, ptx::kStatusTimeout);
                    ok = false;
                    break;
                }
            }
            ok = __all_sync(~0u, ok);
            if (!ok) break;
        }
        const int r0 = chunk * p.rows, r1 = min(r0 + p.rows, s.HW);
        for (int r = r0; r < r1; r += p.srows) {
            ok = __all_sync(~0u, ptx::mbar_wait(ring.empty + stage * 8, phase, &none, a.status, WAIT_LIMIT));
            if (!ok) break;
            const int n = min(p.srows, r1 - r);
            if (r == r0) {  // the statistics that the unit needs
                float2* st = reinterpret_cast<float2*>(ring.smem + stage * p.stage + MAPS * p.data);
                for (int g = lane; g < s.groups; g += 32) {
                    if (MAPS == 2) {
                        const float* q = stats + ((size_t)set * s.groups + g) * 2;
                        st[g] = make_float2(__ldg(q), __ldg(q + 1));
                    }
                    if (pass == 1)
                        st[(MAPS - 1) * s.groups + g] =
                            __ldcg(a.sets + (MAPS == 2 ? (size_t)s.B * s.C : 0) + (size_t)set * s.groups + g);
                }
            }
            __syncwarp();
            if (lane == 0) {
                ring.headers[stage] = Header{pass, set, chunk, r, n, r == r0, r + p.srows >= r1};
                const uint32_t bytes = n * row, dst = ring.base + stage * p.stage, bar = ring.full + stage * 8;
                ptx::mbar_arrive_expect_tx(bar, MAPS * bytes);
                const size_t at = ((size_t)set * s.HW + r) * s.C;
                ptx::bulk_load(dst, x + at, bytes, bar);
                if (MAPS == 2) ptx::bulk_load(dst + p.data, gy + at, bytes, bar);
            }
            __syncwarp();
            if (++stage == p.stages) stage = 0, phase ^= 1;
        }
    }
    // the end, in a stage of its own
    ptx::mbar_wait(ring.empty + stage * 8, phase, &none, a.status, WAIT_LIMIT);
    if (lane == 0) {
        ring.headers[stage].pass = -1;
        ptx::mbar_arrive(ring.full + stage * 8);
    }
}

__device__ __forceinline__ Ring ring_of(uint8_t* smem, Header* headers, uint64_t* bars, int warps) {
    Ring r;
    r.smem = smem;
    r.base = ptx::smem_u32(smem);
    r.headers = headers;
    r.full = ptx::smem_u32(bars);
    r.empty = r.full + MAX_STAGES * 8;
    if (threadIdx.x == 0) {
        for (int i = 0; i < MAX_STAGES; ++i) {
            ptx::mbar_init(r.full + i * 8, 1);
            ptx::mbar_init(r.empty + i * 8, warps);
        }
        ptx::fence_mbar_init();
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return r;
}

// Two sums a channel of the computing threads' u and d, to red[2][slots][C]; returns slots.
template <int P, int NC>
__device__ __forceinline__ int spread(F2 (&u)[P], F2 (&d)[P], int tx, int ty, int cx, int ry, int C, float* red) {
    const bool pow2 = (tx & (tx - 1)) == 0 && tx < 32;
    if (pow2)
        for (int o = tx; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                u[i] = u[i] + shfl_xor(u[i], o);
                d[i] = d[i] + shfl_xor(d[i], o);
            }
    const int slot = pow2 ? (int)threadIdx.x / 32 : ry, slots = pow2 ? NC / 32 : ty;
    if (pow2 ? (int)(threadIdx.x % 32) < tx : ry < ty)
#pragma unroll
        for (int i = 0; i < P; ++i) {
            *reinterpret_cast<F2*>(&red[slot * C + (cx * P + i) * 2]) = u[i];
            *reinterpret_cast<F2*>(&red[(slots + slot) * C + (cx * P + i) * 2]) = d[i];
        }
    return slots;
}

// After a unit's pieces are written: true in the block that finished its set.
template <int NC>
__device__ __forceinline__ bool last_of_set(const Args& a, int set, int* flag) {
    sync_computing<NC>();
    if (threadIdx.x == 0) {
        __threadfence();
        *flag = atomicAdd(a.done + set, 1) == a.p.chunks - 1;
        __threadfence();
    }
    sync_computing<NC>();
    return *flag;
}

template <int NC>
__device__ __forceinline__ void release_set(const Args& a, int set) {
    sync_computing<NC>();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicExch(a.ready + set, 1);
    }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(NC_FWD + 32, 1)
    stream_forward_kernel(const Args a, const T* __restrict__ x, const T* __restrict__ gamma, const T* __restrict__ beta,
                          T* __restrict__ y, float* __restrict__ stats) {
    constexpr int V = 16 / (int)sizeof(T), P = V / 2, NC = NC_FWD, WARPS = NC / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[2 * MAX_STAGES];
    __shared__ Header headers[MAX_STAGES];
    __shared__ int flag;
    const Ring ring = ring_of(smem, headers, bars, NC / 32);
    if (threadIdx.x >= NC) {
        produce<T, 1>(a, ring, x, (const T*)nullptr, nullptr, true);
        return;
    }
    const NormShape& s = a.s;
    const StreamPlan& p = a.p;
    float* red = reinterpret_cast<float*>(smem + p.stages * p.stage);
    const int cg = s.C / s.groups, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int tx = s.C / V, ty = NC / tx, cx = threadIdx.x % tx, ry = threadIdx.x / tx;
    const bool in = ry < ty;
    // k: minus the unit's first pixel, or minus the mean; u, d: the sums, or rstd gamma and beta
    F2 k[P] = {}, u[P] = {}, d[P] = {};
    float* first = red + 2 * NC * V;  // [C] the unit's first pixel
    volatile int none = 0;
    int stage = 0;
    uint32_t phase = 0;
    for (;;) {
        if (!ptx::mbar_wait(ring.full + stage * 8, phase, &none, a.status, WAIT_LIMIT)) break;
        const Header hd = headers[stage];
        if (hd.pass < 0) break;
        const uint4* q = reinterpret_cast<const uint4*>(smem + stage * p.stage) + cx;
        if (hd.pass == 0) {
            if (hd.first) {
                unpack(k, q[0]);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    if (ry == 0) *reinterpret_cast<F2*>(&first[(cx * P + i) * 2]) = k[i];
                    k[i] = k[i] * f2(-1.f);
                    u[i] = d[i] = f2(0.f);
                }
            }
            if (in)
#pragma unroll 4
                for (int r = ry; r < hd.n; r += ty) {
                    F2 v[P];
                    unpack(v, q[r * tx]);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const F2 e = v[i] + k[i];
                        u[i] = u[i] + e;
                        d[i] = fma(e, e, d[i]);
                    }
                }
        } else {
            if (hd.first) {
                const float2* st = reinterpret_cast<const float2*>(smem + stage * p.stage + p.data);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const int c = (cx * P + i) * 2;
                    const float2 v = st[c / cg], w = st[(c + 1) / cg];
                    k[i] = f2(-v.x, -w.x);
                    u[i] = f2(v.y * (gamma ? ld1(gamma + c) : 1.f), w.y * (gamma ? ld1(gamma + c + 1) : 1.f));
                    d[i] = f2(beta ? ld1(beta + c) : 0.f, beta ? ld1(beta + c + 1) : 0.f);
                }
            }
            if (in) {
                T* yp = y + ((size_t)hd.set * s.HW + hd.row0) * s.C + cx * V;
#pragma unroll 4
                for (int r = ry; r < hd.n; r += ty) {
                    F2 v[P];
                    unpack(v, q[r * tx]);
#pragma unroll
                    for (int i = 0; i < P; ++i) v[i] = act_apply<ACT, kFast<T>>(fma(v[i] + k[i], u[i], d[i]));
                    *reinterpret_cast<uint4*>(yp + (size_t)r * s.C) = pack(v);
                }
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ring.empty + stage * 8);
        if (++stage == p.stages) stage = 0, phase ^= 1;
        if (hd.pass == 0 && hd.last) {
            const int slots = spread<P, NC>(u, d, tx, ty, cx, ry, s.C, red);
            sync_computing<NC>();
            const float n = (float)(min((hd.chunk + 1) * p.rows, s.HW) - hd.chunk * p.rows);
            for (int c = threadIdx.x; c < s.C; c += NC) {
                float e = 0.f, f = 0.f;
#pragma unroll 8
                for (int r = 0; r < slots; ++r) {
                    e += red[r * s.C + c];
                    f += red[(slots + r) * s.C + c];
                }
                const float m = e / n, m2 = f - e * m;  // about the first pixel
                red[c] = first[c] + m;
                red[slots * s.C + c] = m2 < 0.f ? 0.f : m2;  // a NaN stays one
            }
            sync_computing<NC>();
            for (int g = warp; g < s.groups; g += WARPS) {
                float e = 0.f;
                for (int c = lane; c < cg; c += 32) e += red[g * cg + c];
                const float mean = warp_sum(e) / (float)cg;
                float m2 = 0.f;
                for (int c = lane; c < cg; c += 32) {
                    const float f = red[g * cg + c] - mean;
                    m2 += red[slots * s.C + g * cg + c] + n * f * f;
                }
                m2 = warp_sum(m2);
                if (lane == 0)
                    a.pieces[((size_t)hd.set * p.chunks + hd.chunk) * s.groups + g] = make_float2(mean, m2);
            }
            if (last_of_set<NC>(a, hd.set, &flag)) {
                const float total = (float)s.HW * (float)cg;
                auto count = [&](int i) { return (float)(min((i + 1) * p.rows, s.HW) - i * p.rows) * (float)cg; };
                for (int g = warp; g < s.groups; g += WARPS) {
                    const float2* pc = a.pieces + (size_t)hd.set * p.chunks * s.groups + g;
                    float e = 0.f, m2 = 0.f;
#pragma unroll 4
                    for (int i = lane; i < p.chunks; i += 32) e += __ldcg(pc + (size_t)i * s.groups).x * (count(i) / total);
                    const float mean = warp_sum(e);
#pragma unroll 4
                    for (int i = lane; i < p.chunks; i += 32) {
                        const float2 v = __ldcg(pc + (size_t)i * s.groups);
                        m2 += v.y + count(i) * (v.x - mean) * (v.x - mean);
                    }
                    m2 = warp_sum(m2);
                    if (lane == 0) {
                        const float2 v = make_float2(mean, rsqrtf(m2 / total + s.eps));
                        const size_t o = (size_t)hd.set * s.groups + g;
                        a.sets[o] = v;
                        if (stats) {
                            stats[2 * o] = v.x;
                            stats[2 * o + 1] = v.y;
                        }
                    }
                }
                release_set<NC>(a, hd.set);
            }
        }
    }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(NC_BWD + 32, 1)
    stream_backward_kernel(const Args a, const T* __restrict__ x, const T* __restrict__ gamma,
                           const T* __restrict__ beta, const float* __restrict__ stats, const T* __restrict__ gy,
                           T* __restrict__ gx, float* __restrict__ gg, float* __restrict__ gb) {
    constexpr int V = 16 / (int)sizeof(T), P = V / 2, NC = NC_BWD, WARPS = NC / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[2 * MAX_STAGES];
    __shared__ Header headers[MAX_STAGES];
    __shared__ int flag;
    const Ring ring = ring_of(smem, headers, bars, NC / 32);
    if (threadIdx.x >= NC) {
        produce<T, 2>(a, ring, x, gy, stats, gx != nullptr);
        return;
    }
    const NormShape& s = a.s;
    const StreamPlan& p = a.p;
    float* red = reinterpret_cast<float*>(smem + p.stages * p.stage);
    const int cg = s.C / s.groups, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int tx = s.C / V, ty = NC / tx, cx = threadIdx.x % tx, ry = threadIdx.x / tx;
    const bool in = ry < ty;
    float2* csums = a.sets;                    // [B][C] sums of a sample's channels
    float2* c12 = a.sets + (size_t)s.B * s.C;  // [B][groups] (c1, c2)
    Channels<P> ch = {};
    F2 u[P] = {}, d[P] = {};  // the sums, or -c1 and -c2
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (cx * P + i) * 2;
        ch.ga[i] = f2(gamma ? ld1(gamma + c) : 1.f, gamma ? ld1(gamma + c + 1) : 1.f);
        ch.be[i] = f2(beta ? ld1(beta + c) : 0.f, beta ? ld1(beta + c + 1) : 0.f);
    }
    volatile int none = 0;
    int stage = 0;
    uint32_t phase = 0;
    for (;;) {
        if (!ptx::mbar_wait(ring.full + stage * 8, phase, &none, a.status, WAIT_LIMIT)) break;
        const Header hd = headers[stage];
        if (hd.pass < 0) break;
        const uint4* q = reinterpret_cast<const uint4*>(smem + stage * p.stage) + cx;
        const uint4* h = reinterpret_cast<const uint4*>(smem + stage * p.stage + p.data) + cx;
        if (hd.first) {
            const float2* st = reinterpret_cast<const float2*>(smem + stage * p.stage + 2 * p.data);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int g0 = (cx * P + i) * 2 / cg, g1 = ((cx * P + i) * 2 + 1) / cg;
                const float2 v = st[g0], w = st[g1];
                ch.nmean[i] = f2(-v.x, -w.x);
                ch.rstd[i] = f2(v.y, w.y);
                u[i] = d[i] = f2(0.f);
                if (hd.pass == 1) {
                    const float2 e = st[s.groups + g0], f = st[s.groups + g1];
                    u[i] = f2(-e.x, -f.x);
                    d[i] = f2(-e.y, -f.y);
                }
            }
        }
        if (in) {
            if (hd.pass == 0) {
#pragma unroll 2
                for (int r = ry; r < hd.n; r += ty) {
                    F2 v[P], g[P], dz[P], hat[P];
                    unpack(v, q[r * tx]);
                    unpack(g, h[r * tx]);
                    ch.template dz<ACT, kFast<T>>(v, g, dz, hat);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        u[i] = u[i] + dz[i];
                        d[i] = fma(dz[i], hat[i], d[i]);
                    }
                }
            } else {
                T* gp = gx + ((size_t)hd.set * s.HW + hd.row0) * s.C + cx * V;
#pragma unroll 2
                for (int r = ry; r < hd.n; r += ty) {
                    F2 v[P], g[P], dz[P], hat[P];
                    unpack(v, q[r * tx]);
                    unpack(g, h[r * tx]);
                    ch.template dz<ACT, kFast<T>>(v, g, dz, hat);
#pragma unroll
                    for (int i = 0; i < P; ++i) v[i] = ch.rstd[i] * fma(hat[i], d[i], fma(ch.ga[i], dz[i], u[i]));
                    *reinterpret_cast<uint4*>(gp + (size_t)r * s.C) = pack(v);
                }
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ring.empty + stage * 8);
        if (++stage == p.stages) stage = 0, phase ^= 1;
        if (hd.pass == 0 && hd.last) {
            const int slots = spread<P, NC>(u, d, tx, ty, cx, ry, s.C, red);
            sync_computing<NC>();
            for (int c = threadIdx.x; c < s.C; c += NC) {
                float e = 0.f, f = 0.f;
#pragma unroll 8
                for (int r = 0; r < slots; ++r) {
                    e += red[r * s.C + c];
                    f += red[(slots + r) * s.C + c];
                }
                a.pieces[((size_t)hd.set * p.chunks + hd.chunk) * s.C + c] = make_float2(e, f);
            }
            if (last_of_set<NC>(a, hd.set, &flag)) {
                for (int c = threadIdx.x; c < s.C; c += NC) {
                    float2 v = make_float2(0.f, 0.f);
#pragma unroll 8
                    for (int i = 0; i < p.chunks; ++i) {
                        const float2 w = __ldcg(a.pieces + ((size_t)hd.set * p.chunks + i) * s.C + c);
                        v.x += w.x;
                        v.y += w.y;
                    }
                    csums[(size_t)hd.set * s.C + c] = v;
                    const float k = gamma ? ld1(gamma + c) : 1.f;
                    red[c] = k * v.x;
                    red[s.C + c] = k * v.y;
                }
                sync_computing<NC>();
                const float inv = 1.f / ((float)s.HW * (float)cg);
                for (int g = warp; g < s.groups; g += WARPS) {
                    float e = 0.f, f = 0.f;
                    for (int c = g * cg + lane; c < (g + 1) * cg; c += 32) {
                        e += red[c];
                        f += red[s.C + c];
                    }
                    e = warp_sum(e);
                    f = warp_sum(f);
                    if (lane == 0) c12[(size_t)hd.set * s.groups + g] = make_float2(e * inv, f * inv);
                }
                release_set<NC>(a, hd.set);
                if (gg || gb) {  // the last set of all sums the parameters' gradients
                    if (threadIdx.x == 0) {
                        flag = atomicAdd(a.finished, 1) == s.B - 1;
                        __threadfence();
                    }
                    sync_computing<NC>();
                    if (flag)
                        for (int c = threadIdx.x; c < s.C; c += NC) params_of(s, csums, c, gg, gb);
                }
            }
        }
    }
}

template <typename F, typename... Q>
cudaError_t launch(F f, DeviceFlags& flags, int threads, const Args& a, cudaStream_t st, Q... args) {
    const uint32_t bytes = a.p.stages * a.p.stage + RED_BYTES + MAX_C * 4;
    cudaError_t e = max_dynamic_smem_once((const void*)f, RING + RED_BYTES + MAX_C * 4, flags);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.p.grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, f, a, args...);
}

cudaError_t args_of(const NormShape& s, const StreamPlan& p, bool backward, void* ws, unsigned* status, cudaStream_t st,
                    Args& a) {
    const Space w = space_of(s, p, backward);
    uint8_t* base = static_cast<uint8_t*>(ws);
    a.s = s;
    a.p = p;
    a.ticket = reinterpret_cast<int*>(base);
    a.finished = a.ticket + 1;
    a.done = a.ticket + 2;
    a.ready = a.done + s.B;
    a.pieces = reinterpret_cast<float2*>(base + w.pieces);
    a.sets = reinterpret_cast<float2*>(base + w.sets);
    a.status = status;
    return cudaMemsetAsync(a.ticket, 0, (2 + 2 * (size_t)s.B) * sizeof(int), st);
}

template <typename T>
cudaError_t forward_t(const Args& a, const T* x, const T* gamma, const T* beta, T* y, float* stats, cudaStream_t st) {
    return with_act(a.s.act, [&](auto A) {
        static DeviceFlags flags;
        return launch(stream_forward_kernel<T, decltype(A)::value>, flags, NC_FWD + 32, a, st, x, gamma, beta, y, stats);
    });
}

template <typename T>
cudaError_t backward_t(const Args& a, const T* x, const T* gamma, const T* beta, const float* stats, const T* gy, T* gx,
                       float* gg, float* gb, cudaStream_t st) {
    return with_act(a.s.act, [&](auto A) {
        static DeviceFlags flags;
        return launch(stream_backward_kernel<T, decltype(A)::value>, flags, NC_BWD + 32, a, st, x, gamma, beta, stats, gy, gx,
                      gg, gb);
    });
}

}  // namespace

bool norm_stream_supported(const NormShape& s, int bf, bool backward) {
    return stream_plan(s, bf ? 2 : 4, backward ? 2 : 1).ok;
}

size_t norm_stream_workspace(const NormShape& s, int bf, bool backward) {
    return space_of(s, stream_plan(s, bf ? 2 : 4, backward ? 2 : 1), backward).total;
}

cudaError_t norm_stream_forward(const NormShape& s, int bf, const void* x, const void* gamma, const void* beta, void* y,
                                float* stats, void* ws, unsigned* status, cudaStream_t st) {
    Args a;
    const cudaError_t e = args_of(s, stream_plan(s, bf ? 2 : 4, 1), false, ws, status, st, a);
    if (e != cudaSuccess) return e;
    return bf ? forward_t(a, (const bf16*)x, (const bf16*)gamma, (const bf16*)beta, (bf16*)y, stats, st)
              : forward_t(a, (const float*)x, (const float*)gamma, (const float*)beta, (float*)y, stats, st);
}

cudaError_t norm_stream_backward(const NormShape& s, int bf, const void* x, const void* gamma, const void* beta,
                                 const float* stats, const void* gy, void* gx, float* gg, float* gb, void* ws,
                                 unsigned* status, cudaStream_t st) {
    Args a;
    const cudaError_t e = args_of(s, stream_plan(s, bf ? 2 : 4, 2), true, ws, status, st, a);
    if (e != cudaSuccess) return e;
    return bf ? backward_t(a, (const bf16*)x, (const bf16*)gamma, (const bf16*)beta, stats, (const bf16*)gy, (bf16*)gx,
                           gg, gb, st)
              : backward_t(a, (const float*)x, (const float*)gamma, (const float*)beta, stats, (const float*)gy,
                           (float*)gx, gg, gb, st);
}

}  // namespace dcn
