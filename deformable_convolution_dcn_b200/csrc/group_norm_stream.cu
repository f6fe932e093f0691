// Group normalisation with an activation, channels last, for long maps of whole
// vectors: a queue of units as in group_norm.cu (all summed first, then applied; what
// L2 still holds by then is not read again from HBM), with the loads taken off the
// threads that compute.
//
// One block an SM. A producer warp claims the units and copies their pixels, in runs
// of one stage, to a ring of shared-memory stages (bulk copies, up to 160 KB in
// flight); most warps compute from there and store; four more warps count the summed
// units and join their sets. So the memory works on while sums are counted, joined and
// released, and those latencies cost little: with the fence and the atomic in a
// computing warp a unit cost nine microseconds more, in a kernel without the ring
// (group_norm.cu) 8x200x200x128 takes 92 us. bfloat16 8x200x200x128 silu takes 59 us,
// 8x100x100x256 relu backward 68.5, with 36 to 46 % of the issue slots and about as much
// of HBM's rate used: the rest is waiting, of the second pass for all sums, and of one
// block an SM for its own joins. The producer waits for a set's statistics
// before it copies a unit of the second pass, and leaves them in its first stage.
//
// A claimed unit waits for none but lower ones, which are summed by blocks that
// never wait (see group_norm.cu), and the warps that join wait for no unit. Every wait
// is bounded; when one runs out, the block's warps leave and the status word says so.
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "kernels.h"
#include "norm.cuh"
#include "tc_ptx.cuh"

namespace dcn {
namespace {

// computing threads: the backward keeps twice the parameters in registers
constexpr int NC_FWD = 608, NC_BWD = 448;
constexpr int JOINERS = 128;             // threads that join, after the producer warp
constexpr int MAX_STAGES = 16;
constexpr int MAX_C = 1024;
constexpr int MAX_GROUPS = 256;          // their statistics travel in a stage
constexpr uint32_t RING = 168 * 1024;    // all stages
constexpr uint32_t RED_BYTES = 2 * NC_FWD * 8 * 4;
#ifndef DCN_NORM_WAIT_LIMIT  // cycles; a test's build sets fewer
#define DCN_NORM_WAIT_LIMIT 2000000000LL
#endif
constexpr long long WAIT_LIMIT = DCN_NORM_WAIT_LIMIT;
constexpr int RUN_STAGES = kRun / 2;     // the backward's stages hold two pixels a thread

struct StreamPlan {
    bool ok;
    int chunks, blocks;    // units of a set (a sample), runs of srows pixels: unit i has the runs i, i + chunks, ...
    int srows, stages;     // pixels a stage, stages
    uint32_t data, stage;  // bytes of one map's pixels, of a stage
    int grid;
};

StreamPlan stream_plan(const NormShape& s, int es, int maps) {
    StreamPlan p = {};
    const int vec = 16 / es, row = s.C * es;
    if (s.C % vec || s.C > MAX_C || s.groups > MAX_GROUPS) return p;
    const int ty = (maps == 1 ? NC_FWD : NC_BWD) / (s.C / vec);
    // four vectors a thread
    p.srows = std::min(4 / maps * ty, s.HW);
    p.data = (uint32_t)p.srows * row;
    p.stage = (maps * (p.data + s.groups * 8) + 127) / 128 * 128;
    p.stages = (int)std::min<uint32_t>(MAX_STAGES, RING / p.stage);
    // A unit costs a few microseconds beside its pixels (reduction, join, wait), so the sets are cut in as many units as
    // there are SMs. Twice as many, of which L2 holds more until their second pass, are better or worse by the activation:
    // backward 8x100x100x256 51.7 us (twice the units: 56.8) without one, 68.5 (63) with relu; forward 8x200x200x128 51.7
    // (49.6) without, 59.6 (54.2) with silu.
    const int chunks = s.B <= 74 ? 148 / s.B : s.B < 148 ? 2 : 1;
    p.blocks = (s.HW + p.srows - 1) / p.srows;
    p.chunks = std::min(chunks, p.blocks);
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
constexpr int kPut = 16, kAdd = 32, kTake = 64;
struct __align__(16) Header {
    int pass;   // 0 sums, 1 applies, -1: no more units; + 4: the first stage of a run, the unit's statistics in it; + 8:
                // the unit's last. + kPut: the sums of the run before are put by, + kAdd: with others that were; + kTake: and
                // taken for the unit's
    int set, chunk;
    int row0;   // its pixels, srows or up to the end of the sample
};

// The queue: every set's units summed, then every set's applied.
__device__ __forceinline__ void unit_at(const Args& a, int t, int& pass, int& set, int& chunk) {
    const int half = a.s.B * a.p.chunks;
    pass = t >= half;
    set = (t - pass * half) / a.p.chunks;
    chunk = t % a.p.chunks;
}

// Pixels of a set's unit i.
__device__ __forceinline__ int pixels_of(const Args& a, int i) {
    const int more = (a.p.blocks - 1) / a.p.chunks, last = a.p.blocks - 1 - more * a.p.chunks;
    return (more + (i <= last)) * a.p.srows - (i == last ? a.p.blocks * a.p.srows - a.s.HW : 0);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Waits, a warp, until the set's sums are joined; false when the bounded wait ran out.
__device__ __forceinline__ bool await_set(const Args& a, int set) {
    bool ok = true;
    if (ptx::ld_acquire_gpu(a.ready + set) == 0) {
        const long long t0 = clock64();
        while (ptx::ld_acquire_gpu(a.ready + set) == 0) {
            __nanosleep(100);
            if (clock64() - t0 > WAIT_LIMIT) {
                atomicOr(a.status, ptx::kStatusTimeout);
                ok = false;
                break;
            }
        }
    }
    return __all_sync(~0u, ok);
}

struct Ring {
    uint8_t* smem;
    uint32_t base, full, empty;  // shared addresses: stages, barriers
    Header* headers;
    // summed units on their way to the joining warps, in two slots: the set (-1: no more), its barriers
    int* unit_set;
    uint32_t unit_done, unit_free;
    volatile int* aborted;  // a wait of the block ran out: every warp leaves
};

// Warps that wait by themselves for the same things (the computing warps, the joining warps) leave together when a wait of
// one of them ran out: none stays behind at a barrier. A warp whose wait failed goes to the next agreement at once, the
// others when they come there, all within bounded time: the first barrier behind a wait is always one, and so is every way
// out of their loops. (Warps that leave alone, with barriers that give up, cost 5 % of 8x200x200x128; with a look at a flag
// behind every barrier, 7 % of 4096x7x7x256.)
constexpr int COMPUTING = 1, JOINING = 2;  // named barriers
template <int ID, int THREADS>
__device__ __forceinline__ bool agree_to_leave(bool failed) {
    return ptx::bar_or_named(ID, THREADS, failed);
}

template <int NC>
__device__ __forceinline__ void sync_computing() {
    ptx::bar_sync_named(COMPUTING, NC);
}
__device__ __forceinline__ void sync_joiners() { ptx::bar_sync_named(JOINING, JOINERS); }

// The producer warp. MAPS: x, or x and grad_y; stats: the backward's (mean, rstd); apply: the second pass is wanted.
template <typename T, int MAPS>
__device__ __forceinline__ void produce(const Args& a, const Ring& ring, const T* x, const T* gy, const float* stats,
                                        bool apply) {
    const NormShape& s = a.s;
    const StreamPlan& p = a.p;
    const int lane = threadIdx.x % 32;
    const int total = (apply ? 2 : 1) * s.B * p.chunks;
    const uint32_t row = s.C * (uint32_t)sizeof(T);
    int stage = 0, copied = 0;
    uint32_t phase = 1;
    bool ok = true;
    // Claimed when the unit before is on its way, not earlier: the ring hides the answer's time, and a unit held by a
    // block that is not at it is one that an idle block misses.
    for (;;) {
        int t = 0;
        if (lane == 0) t = atomicAdd(a.ticket, 1);
        t = __shfl_sync(~0u, t, 0);
        if (t >= total || !ok) break;
        int pass, set, chunk;
        unit_at(a, t, pass, set, chunk);
        if (pass == 1) {  // the set's sums are joined
            ok = await_set(a, set);
            if (!ok) break;
        }
        int j = 0;  // the unit's stage
        for (int k = chunk; k < p.blocks; k += p.chunks, ++j) {
            const int r = k * p.srows;
            ok = __all_sync(~0u, ptx::mbar_wait(ring.empty + stage * 8, phase, ring.aborted, a.status, WAIT_LIMIT));
            if (!ok) break;
            const int n = min(p.srows, s.HW - r);
            // the backward's first pass goes by runs (see kRun)
            const int before = MAPS == 2 && pass == 0 ? j / RUN_STAGES : 0;
            const bool first = j == before * RUN_STAGES, last = k + p.chunks >= p.blocks;
            if (first) {  // the statistics that the unit needs
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
                const int flags = (first ? 4 : 0) | (last ? 8 : 0) | (first && before > 0 ? kPut : 0) |
                                  (first && before > 1 ? kAdd : 0) | (last && before > 0 ? kTake : 0);
                ring.headers[stage] = Header{pass | flags, set, chunk, r};
                const uint32_t bytes = n * row, dst = ring.base + stage * p.stage, bar = ring.full + stage * 8;
                ptx::mbar_arrive_expect_tx(bar, MAPS * bytes);
                const size_t at = ((size_t)set * s.HW + r) * s.C;
                ptx::bulk_load(dst, x + at, bytes, bar);
                if (MAPS == 2) ptx::bulk_load(dst + p.data, gy + at, bytes, bar);
            }
            __syncwarp();
            ++copied;
            if (++stage == p.stages) stage = 0, phase ^= 1;
        }
    }
    // the end, in a stage of its own
    ok = __all_sync(~0u, ptx::mbar_wait(ring.empty + stage * 8, phase, ring.aborted, a.status, WAIT_LIMIT));
    if (lane == 0) {
        if (ok) {
            ring.headers[stage].pass = -1;
            ptx::mbar_arrive(ring.full + stage * 8);
        }
        // copies still in flight land before the block may end (that of the end's stage has: the stage was free)
        volatile int none = 0;
        for (int k = max(0, copied - p.stages + (ok ? 1 : 0)); k < copied; ++k)
            ptx::mbar_wait(ring.full + (k % p.stages) * 8, (k / p.stages) & 1, &none, nullptr, WAIT_LIMIT);
    }
    __syncwarp();
}

__device__ __forceinline__ Ring ring_of(uint8_t* smem, Header* headers, uint64_t* bars, int* unit_set, int* aborted,
                                        int warps) {
    Ring r;
    r.smem = smem;
    r.base = ptx::smem_u32(smem);
    r.headers = headers;
    r.full = ptx::smem_u32(bars);
    r.empty = r.full + MAX_STAGES * 8;
    r.unit_set = unit_set;
    r.unit_done = r.empty + MAX_STAGES * 8;
    r.unit_free = r.unit_done + 16;
    r.aborted = aborted;
    if (threadIdx.x == 0) {
        *aborted = 0;
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(r.unit_done + i * 8, warps);
            ptx::mbar_init(r.unit_free + i * 8, 1);
        }
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

// As spread, of moments: minus the levels (means) k, the squares about them d and the number of values n of each thread,
// to red[2][slots][C] and counts[slots].
template <int P, int NC>
__device__ __forceinline__ int spread_moments(F2 (&k)[P], F2 (&d)[P], int n, int tx, int ty, int cx, int ry, int C,
                                              float* red, float* counts) {
    const bool pow2 = (tx & (tx - 1)) == 0 && tx < 32;
    if (pow2)
        for (int o = tx; o < 32; o <<= 1) {
            const int nb = __shfl_xor_sync(~0u, n, o);
            // the parts' weights: the mean moves by e nb / (n + nb), the squares grow by e^2 n nb / (n + nb)
            const float w = (float)nb * rcp_fast((float)max(n + nb, 1));  // (a division took 1.5 us of 8x200x200x128)
            const F2 wb = f2(w), wq = f2((float)n * w);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const F2 e = shfl_xor(k[i], o) + k[i] * f2(-1.f);
                d[i] = fma(e * e, wq, d[i] + shfl_xor(d[i], o));
                k[i] = fma(e, wb, k[i]);
            }
            n += nb;
        }
    const int slot = pow2 ? (int)threadIdx.x / 32 : ry, slots = pow2 ? NC / 32 : ty;
    if (pow2 ? (int)(threadIdx.x % 32) < tx : ry < ty) {
        if (cx == 0) counts[slot] = (float)n;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            *reinterpret_cast<F2*>(&red[slot * C + (cx * P + i) * 2]) = k[i] * f2(-1.f);
            *reinterpret_cast<F2*>(&red[(slots + slot) * C + (cx * P + i) * 2]) = d[i];
        }
    }
    return slots;
}

// The sums of a unit's runs before the one under way: to the thread's places of red, which is free until the unit's end
// (u and d), or added to u and d from there.
template <int P, int NC>
__device__ __forceinline__ void runs_sums(F2 (&u)[P], F2 (&d)[P], float* red, bool take) {
    const uint32_t mine = ptx::smem_u32(red) + threadIdx.x * 16;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (take) {
            F2 v[2];
            unpack(v, ptx::lds_v4(mine + i * (NC * 16)));
            u[i] = u[i] + v[0];
            d[i] = d[i] + v[1];
        } else {
            const F2 v[2] = {u[i], d[i]};
            ptx::sts_v4(mine + i * (NC * 16), pack(v));
        }
    }
}

// The computing warps' side of the way to the joining warps.
struct Post {
    int n = 0;
    // The unit's pieces are written by this thread; set -1: no more units. All computing threads.
    __device__ __forceinline__ void operator()(const Args& a, const Ring& ring, int set) {
        const int slot = n & 1;
        if (threadIdx.x == 0) {  // the slot's unit before the last has been taken
            if (n >= 2) ptx::mbar_wait(ring.unit_free + slot * 8, ((n >> 1) - 1) & 1, ring.aborted, a.status, WAIT_LIMIT);
            ring.unit_set[slot] = set;
        }
        __syncwarp();
        if (threadIdx.x % 32 == 0) ptx::mbar_arrive(ring.unit_done + slot * 8);
        ++n;
    }
};

// The joining warps: counts each summed unit in its set, and join(set) for the sets that this block has finished.
template <typename F>
__device__ __forceinline__ void join_sets(const Args& a, const Ring& ring, int* flag, F&& join) {
    const bool head = threadIdx.x % 32 == 0 && (int)threadIdx.x == (int)blockDim.x - JOINERS;
    for (int n = 0;; ++n) {
        const int slot = n & 1;
        // a unit may be a long time away, the wait of the producer among the reasons
        const bool ok = __all_sync(
            ~0u, ptx::mbar_wait(ring.unit_done + slot * 8, (n >> 1) & 1, ring.aborted, a.status, 4 * WAIT_LIMIT));
        const int set = ring.unit_set[slot];
        if (agree_to_leave<JOINING, JOINERS>(!ok || set < 0)) return;
        if (head) {
            ptx::mbar_arrive(ring.unit_free + slot * 8);
            __threadfence();
            *flag = atomicAdd(a.done + set, 1) == a.p.chunks - 1;
            __threadfence();
        }
        sync_joiners();
        if (*flag) {
            join(set);
            sync_joiners();  // all of it is written
            if (head) {
                __threadfence();
                atomicExch(a.ready + set, 1);
            }
        }
    }
}

// The forward's join: mean and rstd of a set's groups. Four threads share a group's units, each with sums about a level
// that moves to the mean after every batch of them (see Running).
__device__ __forceinline__ void join_stats(const Args& a, int set, float* stats, float4* sm) {
    const NormShape& s = a.s;
    const StreamPlan& p = a.p;
    const int t = threadIdx.x - (blockDim.x - JOINERS), cg = s.C / s.groups;
    const float inv = 1.f / ((float)s.HW * (float)cg);
    // values of a group in the units before, at and behind the one with the last run
    const int most = (p.blocks - 1) / p.chunks, last = p.blocks - 1 - most * p.chunks;
    const float before = (float)((most + 1) * p.srows) * (float)cg, behind = (float)(most * p.srows) * (float)cg;
    const float at = (float)pixels_of(a, last) * (float)cg;
    for (int base = 0; base < s.groups; base += 32) {
        const int g = base + t % 32, part = t / 32;
        float u = 0.f, m2 = 0.f, n = 0.f, level = 0.f;
        if (g < s.groups && part < p.chunks) {
            const float2* pc = a.pieces + (size_t)set * p.chunks * s.groups + g;
            constexpr int STEP = JOINERS / 32, BATCH = 10;  // (units of a batch of eight samples: 18, 5 a thread)
            for (int i0 = part; i0 < p.chunks; i0 += BATCH * STEP) {
                float2 v[BATCH];  // all loads in flight
#pragma unroll
                for (int j = 0; j < BATCH; ++j)
                    if (i0 + j * STEP < p.chunks) v[j] = __ldcg(pc + (size_t)(i0 + j * STEP) * s.groups);
                if (i0 == part) level = v[0].x;
#pragma unroll
                for (int j = 0; j < BATCH; ++j)
                    if (i0 + j * STEP < p.chunks) {
                        const int i = i0 + j * STEP;
                        const float c = i < last ? before : i == last ? at : behind, d = v[j].x - level;
                        n += c;
                        u = fmaf(c, d, u);
                        m2 += fmaf(c * d, d, v[j].y);
                    }
                const float m = u * rcp_fast(n);
                m2 = fmaf(-u, m, m2);
                level += m;
                u = 0.f;
            }
        }
        sm[t] = make_float4(n, level, m2, 0.f);
        sync_joiners();
        if (part == 0 && g < s.groups) {
            float4 v[JOINERS / 32];
            float e = 0.f, var = 0.f;
#pragma unroll
            for (int k = 0; k < JOINERS / 32; ++k) {
                v[k] = sm[k * 32 + t];
                if (v[k].x > 0.f) e = fmaf(v[k].x * inv, v[k].y - level, e);
            }
            level += e;
#pragma unroll
            for (int k = 0; k < JOINERS / 32; ++k)
                if (v[k].x > 0.f) var += fmaf(v[k].x * (v[k].y - level), v[k].y - level, v[k].z) * inv;
            const float2 out = make_float2(level, rsqrtf((var < 0.f ? 0.f : var) + s.eps));
            const size_t o = (size_t)set * s.groups + g;
            a.sets[o] = out;
            if (stats) {
                stats[2 * o] = out.x;
                stats[2 * o + 1] = out.y;
            }
        }
        sync_joiners();
    }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(NC_FWD + 32 + JOINERS, 1)
    stream_forward_kernel(const Args a, const T* __restrict__ x, const T* __restrict__ gamma, const T* __restrict__ beta,
                          T* __restrict__ y, float* __restrict__ stats) {
    constexpr int V = 16 / (int)sizeof(T), P = V / 2, NC = NC_FWD, WARPS = NC / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[2 * MAX_STAGES + 4];
    __shared__ int unit_set[2], aborted;
    __shared__ Header headers[MAX_STAGES];
    __shared__ int flag;
    __shared__ float4 scratch[JOINERS];
    const Ring ring = ring_of(smem, headers, bars, unit_set, &aborted, NC / 32);
    if (threadIdx.x >= NC + 32) {
        join_sets(a, ring, &flag, [&](int set) { join_stats(a, set, stats, scratch); });
        return;
    }
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
    // each channel's group (a division each, otherwise, for every unit)
    uint16_t* group = reinterpret_cast<uint16_t*>(smem + p.stages * p.stage + RED_BYTES + MAX_C * 4);
    for (int c = threadIdx.x; c < s.C; c += NC) group[c] = (uint16_t)(c / cg);
    sync_computing<NC>();
    // summing: see Running; applying: k minus the mean, u rstd gamma, d beta
    Running<P> m = {};
    auto &k = m.k, &u = m.u, &d = m.d;
    int stages = 0, next = 1;         // of the unit, and at which the level moves
    const int each = in && ry < p.srows ? (p.srows - 1 - ry) / ty + 1 : 0;  // this thread's pixels of a whole stage
    float* counts = red + 2 * NC * V;  // [slots] values of a slot
    Post post;
    int stage = 0;
    uint32_t phase = 0;
    for (;;) {
        const bool there =
            __all_sync(~0u, ptx::mbar_wait(ring.full + stage * 8, phase, ring.aborted, a.status, WAIT_LIMIT));
        if (!there || headers[stage].pass < 0) {
            if (agree_to_leave<COMPUTING, NC>(!there)) return;
            break;
        }
        const Header hd = headers[stage];
        const bool apply = hd.pass & 1, first_stage = hd.pass & 4, last_stage = hd.pass & 8;
        const int n = min(p.srows, s.HW - hd.row0);
        const uint4* q = reinterpret_cast<const uint4*>(smem + stage * p.stage) + cx;
        if (!apply) {
            if (first_stage) {
                m.start(q[min(ry, n - 1) * tx]);
                stages = 0;
                next = 1;
            }
            if (in)
#pragma unroll 4
                for (int r = ry; r < n; r += ty) m.add(q[r * tx]);
            if (++stages == next || last_stage) {  // (the stages before a unit's last are whole)
                m.n = (stages - 1) * each + (n == p.srows ? each : in && ry < n ? (n - 1 - ry) / ty + 1 : 0);
                m.level();
                next *= 2;
            }
        } else {
            if (first_stage) {
                const float2* st = reinterpret_cast<const float2*>(smem + stage * p.stage + p.data);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const int c = (cx * P + i) * 2;
                    const float2 v = st[group[c]], w = st[group[c + 1]];
                    k[i] = f2(-v.x, -w.x);
                    u[i] = f2(v.y * (gamma ? ld1(gamma + c) : 1.f), w.y * (gamma ? ld1(gamma + c + 1) : 1.f));
                    d[i] = f2(beta ? ld1(beta + c) : 0.f, beta ? ld1(beta + c + 1) : 0.f);
                }
            }
            if (in) {
                T* yp = y + ((size_t)hd.set * s.HW + hd.row0) * s.C + cx * V;
#pragma unroll 4
                for (int r = ry; r < n; r += ty) {
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
        if (!apply && last_stage) {
            const int slots = spread_moments<P, NC>(k, d, m.n, tx, ty, cx, ry, s.C, red, counts);
            if (agree_to_leave<COMPUTING, NC>(false)) return;
            const float count = (float)pixels_of(a, hd.chunk);
            for (int c = threadIdx.x; c < s.C; c += NC)
                join_slots(red + c, s.C, slots, count, [&](int r) { return counts[r]; });
            sync_computing<NC>();
            for (int g = warp; g < s.groups; g += WARPS) {
                float e = 0.f;
                for (int c = lane; c < cg; c += 32) e += red[g * cg + c];
                const float mean = warp_sum(e) / (float)cg;
                float m2 = 0.f;
                for (int c = lane; c < cg; c += 32) {
                    const float f = red[g * cg + c] - mean;
                    m2 += red[slots * s.C + g * cg + c] + count * f * f;
                }
                m2 = warp_sum(m2);
                if (lane == 0)
                    a.pieces[((size_t)hd.set * p.chunks + hd.chunk) * s.groups + g] = make_float2(mean, m2);
            }
            post(a, ring, hd.set);
            sync_computing<NC>();  // red is free
        }
    }
    post(a, ring, -1);
}

// The backward's join: the sums of a set's channels, c1 and c2 of its groups; after the last set of all, the
// parameters' gradients. sm: [2][MAX_C].
template <typename T>
__device__ __forceinline__ void join_sums(const Args& a, int set, const T* gamma, float* gg, float* gb, float* sm,
                                          int* last) {
    const NormShape& s = a.s;
    const StreamPlan& p = a.p;
    const int t = threadIdx.x - (blockDim.x - JOINERS), warp = t / 32, lane = t % 32, cg = s.C / s.groups;
    float2* csums = a.sets;                    // [B][C] sums of a sample's channels
    float2* c12 = a.sets + (size_t)s.B * s.C;  // [B][groups] (c1, c2)
    for (int c = t; c < s.C; c += JOINERS) {
        float2 v = make_float2(0.f, 0.f);
#pragma unroll 16
        for (int i = 0; i < p.chunks; ++i) {
            const float2 w = __ldcg(a.pieces + ((size_t)set * p.chunks + i) * s.C + c);
            v.x += w.x;
            v.y += w.y;
        }
        csums[(size_t)set * s.C + c] = v;
        const float k = gamma ? ld1(gamma + c) : 1.f;
        sm[c] = k * v.x;
        sm[MAX_C + c] = k * v.y;
    }
    sync_joiners();
    const float inv = 1.f / ((float)s.HW * (float)cg);
    for (int g = warp; g < s.groups; g += JOINERS / 32) {
        float e = 0.f, f = 0.f;
        for (int c = g * cg + lane; c < (g + 1) * cg; c += 32) {
            e += sm[c];
            f += sm[MAX_C + c];
        }
        e = warp_sum(e);
        f = warp_sum(f);
        if (lane == 0) c12[(size_t)set * s.groups + g] = make_float2(e * inv, f * inv);
    }
    if (gg || gb) {
        sync_joiners();
        if (t == 0) {
            __threadfence();
            *last = atomicAdd(a.finished, 1) == s.B - 1;
            __threadfence();
        }
        sync_joiners();
        if (*last)
            for (int c = t; c < s.C; c += JOINERS) params_of(s, csums, c, gg, gb);
    }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(NC_BWD + 32 + JOINERS, 1)
    stream_backward_kernel(const Args a, const T* __restrict__ x, const T* __restrict__ gamma,
                           const T* __restrict__ beta, const float* __restrict__ stats, const T* __restrict__ gy,
                           T* __restrict__ gx, float* __restrict__ gg, float* __restrict__ gb) {
    constexpr int V = 16 / (int)sizeof(T), P = V / 2, NC = NC_BWD;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[2 * MAX_STAGES + 4];
    __shared__ int unit_set[2], aborted;
    __shared__ Header headers[MAX_STAGES];
    __shared__ int flag, last;
    __shared__ float scratch[2 * MAX_C];
    const Ring ring = ring_of(smem, headers, bars, unit_set, &aborted, NC / 32);
    if (threadIdx.x >= NC + 32) {
        join_sets(a, ring, &flag, [&](int set) { join_sums(a, set, gamma, gg, gb, scratch, &last); });
        return;
    }
    if (threadIdx.x >= NC) {
        produce<T, 2>(a, ring, x, gy, stats, gx != nullptr);
        return;
    }
    const NormShape& s = a.s;
    const StreamPlan& p = a.p;
    float* red = reinterpret_cast<float*>(smem + p.stages * p.stage);
    const int cg = s.C / s.groups, lane = threadIdx.x % 32;
    const int tx = s.C / V, ty = NC / tx, cx = threadIdx.x % tx, ry = threadIdx.x / tx;
    const bool in = ry < ty;
    // each channel's group (a division each, otherwise, for every unit)
    uint16_t* group = reinterpret_cast<uint16_t*>(smem + p.stages * p.stage + RED_BYTES + MAX_C * 4);
    for (int c = threadIdx.x; c < s.C; c += NC) group[c] = (uint16_t)(c / cg);
    sync_computing<NC>();
    Post post;
    Channels<P> ch = {};
    F2 u[P] = {}, d[P] = {};  // the sums, or -c1 and -c2
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (cx * P + i) * 2;
        ch.ga[i] = f2(gamma ? ld1(gamma + c) : 1.f, gamma ? ld1(gamma + c + 1) : 1.f);
        ch.be[i] = f2(beta ? ld1(beta + c) : 0.f, beta ? ld1(beta + c + 1) : 0.f);
    }
    ch.set_border();
    int stage = 0;
    uint32_t phase = 0;
    for (;;) {
        const bool there =
            __all_sync(~0u, ptx::mbar_wait(ring.full + stage * 8, phase, ring.aborted, a.status, WAIT_LIMIT));
        if (!there || headers[stage].pass < 0) {
            if (agree_to_leave<COMPUTING, NC>(!there)) return;
            break;
        }
        const Header hd = headers[stage];
        const bool apply = hd.pass & 1, first_stage = hd.pass & 4, last_stage = hd.pass & 8;
        const int n = min(p.srows, s.HW - hd.row0);
        const uint4* q = reinterpret_cast<const uint4*>(smem + stage * p.stage) + cx;
        const uint4* h = reinterpret_cast<const uint4*>(smem + stage * p.stage + p.data) + cx;
        if (first_stage) {
            if (hd.pass & kPut) {
                if (hd.pass & kAdd) runs_sums<P, NC>(u, d, red, true);
                runs_sums<P, NC>(u, d, red, false);
            }
            const float2* st = reinterpret_cast<const float2*>(smem + stage * p.stage + 2 * p.data);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int g0 = group[(cx * P + i) * 2], g1 = group[(cx * P + i) * 2 + 1];
                const float2 v = st[g0], w = st[g1];
                ch.nmean[i] = f2(-v.x, -w.x);
                ch.rstd[i] = f2(v.y, w.y);
                u[i] = d[i] = f2(0.f);
                if (apply) {
                    const float2 e = st[s.groups + g0], f = st[s.groups + g1];
                    u[i] = f2(-e.x, -f.x);
                    d[i] = f2(-e.y, -f.y);
                }
            }
        }
        if (in) {
            if (!apply) {
#pragma unroll 2
                for (int r = ry; r < n; r += ty) {
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
                for (int r = ry; r < n; r += ty) {
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
        if (!apply && last_stage) {
            if (hd.pass & kTake) {
                runs_sums<P, NC>(u, d, red, true);
                if (agree_to_leave<COMPUTING, NC>(false)) return;  // red is the unit's
            }
            const int slots = spread<P, NC>(u, d, tx, ty, cx, ry, s.C, red);
            if (agree_to_leave<COMPUTING, NC>(false)) return;
            for (int c = threadIdx.x; c < s.C; c += NC) {
                float e = 0.f, f = 0.f;
#pragma unroll 8
                for (int r = 0; r < slots; ++r) {
                    e += red[r * s.C + c];
                    f += red[(slots + r) * s.C + c];
                }
                a.pieces[((size_t)hd.set * p.chunks + hd.chunk) * s.C + c] = make_float2(e, f);
            }
            post(a, ring, hd.set);
            sync_computing<NC>();  // red is free
        }
    }
    post(a, ring, -1);
}

template <typename F, typename... Q>
cudaError_t launch(F f, DeviceFlags& flags, int threads, const Args& a, cudaStream_t st, Q... args) {
    const uint32_t bytes = a.p.stages * a.p.stage + RED_BYTES + MAX_C * 6;
    cudaError_t e = max_dynamic_smem_once((const void*)f, RING + RED_BYTES + MAX_C * 6, flags);
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
        return launch(stream_forward_kernel<T, decltype(A)::value>, flags, NC_FWD + 32 + JOINERS, a, st, x, gamma, beta, y, stats);
    });
}

template <typename T>
cudaError_t backward_t(const Args& a, const T* x, const T* gamma, const T* beta, const float* stats, const T* gy, T* gx,
                       float* gg, float* gb, cudaStream_t st) {
    return with_act(a.s.act, [&](auto A) {
        static DeviceFlags flags;
        return launch(stream_backward_kernel<T, decltype(A)::value>, flags, NC_BWD + 32 + JOINERS, a, st, x, gamma, beta, stats, gy, gx,
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

const float2* norm_stream_sums(const NormShape& s, int bf, const void* ws) {
    const Space w = space_of(s, stream_plan(s, bf ? 2 : 4, 2), true);
    return reinterpret_cast<const float2*>(static_cast<const uint8_t*>(ws) + w.sets);
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
