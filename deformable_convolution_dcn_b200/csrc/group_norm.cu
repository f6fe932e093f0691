// Group normalisation with an activation, channels last: for each sample b and
// group g of C / groups channels, over its n = H W C / groups values,
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps),
//   z = gamma (x - mean) rstd + beta,  y = act(z),
// and backward, with xh = (x - mean) rstd and dz = grad_y act'(z),
//   grad_beta = sum_{b,p} dz,  grad_gamma = sum_{b,p} dz xh,
//   c1 = sum_g gamma dz / n,  c2 = sum_g gamma dz xh / n,
//   grad_x = rstd (gamma dz - c1 - xh c2).
//
// Maps whose blocks of channels fit a small cluster's shared memory go to
// group_norm_cluster.cu. The kernels here take every map, in one launch over a
// queue of units. A unit is a run of pixels of one set (a sample's block of
// whole groups); it is met twice, first to sum and then to apply, and the queue
// holds the second pass of a set a few sets behind the first, so that the second
// reads the map from L2: HBM sees it read once and written once. The last unit
// of a set to be summed joins the set's sums (in the order of the units, so that
// equal calls give equal bits) and lets its second pass go.
//
// A block claims its units by an atomic counter, in order. A unit of the second
// pass waits for units ahead of it in the queue alone, so the lowest unfinished
// unit can always run, however many blocks are resident. The waits are bounded; a
// block whose wait ran out takes no more units, and the status word says so.
//
// A thread keeps one 16-byte vector of channels and walks the pixels, eight
// loads in flight. Sums are float32: the statistics are taken about a level that
// follows the mean (Running in norm.cuh) and joined as means and sums of squares
// about them, so that a level far from zero costs no digits, nor does a first pixel
// far from the others.
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "kernels.h"
#include "norm.cuh"
#include "tc_ptx.cuh"

namespace dcn {
namespace {

constexpr int NT = 256;                 // threads a block
constexpr int MAX_COLS = 1024;          // channels a unit at most (V = 1: 256)
constexpr int UNIT_BYTES = 96 * 1024;   // of a map that fills the GPU many times
#ifndef DCN_NORM_WAIT_LIMIT  // cycles; a test's build sets fewer
#define DCN_NORM_WAIT_LIMIT 2000000000LL
#endif
constexpr long long WAIT_LIMIT = DCN_NORM_WAIT_LIMIT;

// How a map is cut. Blocks of cb channels: gpb whole groups, or (gpb = 0) parts
// of one group.
struct Plan {
    int V;         // channels a vector
    int gpb;       // groups a channel block; 0: a group takes `parts` blocks
    int cb;        // channels a block
    int parts;     // blocks a group (gpb = 0), else 1
    int sets;      // sets a sample: blocks of groups, or groups
    int chunks, rows;
    int units;     // units a set: parts * chunks
    int lag;       // sets that the second pass stays behind
    int grid;
};

Plan make_plan(const NormShape& s, int vec, int es, int maps) {
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
        }
    }
    if (p.V == 1) p.gpb = cg <= NT ? std::min(NT / cg, s.groups) : 0;
    if (p.gpb) {
        p.cb = p.gpb * cg;
        p.parts = 1;
        p.sets = (s.groups + p.gpb - 1) / p.gpb;
    } else {
        p.cb = p.V == 1 ? NT : MAX_COLS;
        p.parts = (cg + p.cb - 1) / p.cb;
        p.sets = s.groups;
    }
    const int ty = NT / ((p.cb + p.V - 1) / p.V);
    const long long nsets = (long long)s.B * p.sets;
    p.grid = 148 * (maps == 1 ? 3 : 2);
    // units of UNIT_BYTES, or small enough to give every block one; at least four pixels a thread
    long long rows = std::max<long long>(1, UNIT_BYTES / ((long long)p.cb * es * maps));
    rows = std::min(rows, std::max<long long>(1, (long long)s.HW * nsets * p.parts / p.grid));
    rows = std::max(rows, 4LL * ty);
    rows = std::max(rows, (s.HW + 255LL) / 256);  // the join walks at most 256 chunks
    p.rows = (int)std::min<long long>(rows, s.HW);
    p.chunks = (s.HW + p.rows - 1) / p.rows;
    p.units = p.parts * p.chunks;
    // far enough behind that a set is summed by the time its second pass is claimed
    p.lag = (int)std::min<long long>(nsets, p.grid / p.units + 2);
    p.grid = (int)std::min<long long>(p.grid, nsets * p.units);
    return p;
}

// Workspace: counters (zeroed by each call), then per unit and set.
struct Space {
    size_t counters, pieces, sets, total;  // offsets
};
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
Space space_of(const NormShape& s, const Plan& p, bool backward) {
    Space w;
    const size_t nsets = (size_t)s.B * p.sets;
    w.counters = 0;
    w.pieces = up256((2 + 2 * nsets) * sizeof(int));
    // forward: (mean, m2) of each unit's groups, then (mean, rstd) of each sample's groups;
    // backward: (sum dz, sum dz xh) of each unit's channels, then of each sample's, then (c1, c2) of its groups
    const size_t n = backward ? (size_t)s.B * p.chunks * s.C : (size_t)s.B * p.chunks * s.groups * p.parts;
    w.sets = up256(w.pieces + n * sizeof(float2));
    w.total = up256(w.sets + (size_t)s.B * (backward ? s.C + s.groups : s.groups) * sizeof(float2));
    return w;
}

struct Args {
    NormShape s;
    Plan p;
    int *ticket, *finished, *done, *ready;  // counters: units claimed, sets joined, units summed, sets joined (each)
    float2 *pieces, *sets;
    unsigned* status;
};

// The queue's unit t: the pass (0 sums, 1 applies), set and unit within the set.
__device__ __forceinline__ void unit_at(const Args& a, int t, int& pass, int& set, int& unit) {
    const int U = a.p.units, Q = a.s.B * a.p.sets, L = a.p.lag;
    if (t < L * U) {
        pass = 0;
        set = t / U;
        unit = t % U;
        return;
    }
    int r = t - L * U;
    if (r < (Q - L) * 2 * U) {
        const int i = r / (2 * U), w = r % (2 * U);
        pass = w >= U;
        set = pass ? i : L + i;
        unit = pass ? w - U : w;
        return;
    }
    r -= (Q - L) * 2 * U;
    pass = 1;
    set = Q - L + r / U;
    unit = r % U;
}

// A unit's place: channels [c0, c0 + nc), groups [g0, g0 + ng), pixels [r0, r1) of sample b.
struct Place {
    int b, c0, nc, g0, ng, part, chunk, r0, r1;
};
__device__ __forceinline__ Place place_of(const Args& a, int set, int unit) {
    const NormShape& s = a.s;
    const Plan& p = a.p;
    const int cg = s.C / s.groups, in = set % p.sets;
    Place c;
    c.b = set / p.sets;
    c.part = unit % p.parts;
    c.chunk = unit / p.parts;
    if (p.gpb) {
        c.g0 = in * p.gpb;
        c.ng = min(p.gpb, s.groups - c.g0);
        c.c0 = c.g0 * cg;
        c.nc = c.ng * cg;
    } else {
        c.g0 = in;
        c.ng = 1;
        c.c0 = in * cg + c.part * p.cb;
        c.nc = min(p.cb, cg - c.part * p.cb);
    }
    c.r0 = c.chunk * p.rows;
    c.r1 = min(c.r0 + p.rows, s.HW);
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// A sum written by other blocks (past the L1 cache, which may hold an older line).
__device__ __forceinline__ float2 ld_l2(const float2* p) {
    return __ldcg(p);
}

// The block's way through the queue. Thread 0's atomics are answered while the block works: the claim of the next
// unit is made a unit ahead, and whether a summed unit was its set's last is looked at a unit later.
struct Queue {
    const Args& a;
    int* shared;          // [3]: the unit claimed, the set to join (or -1), whether a wait ran out
    int total;
    int claim = 0;        // thread 0
    int count = 0;        // thread 0: units summed of `set` before the last one summed here
    int set = -1;         // the set of the unit summed last, until that is looked at
    __device__ Queue(const Args& args, int* s) : a(args), shared(s) {
        total = 2 * a.s.B * a.p.sets * a.p.units;
        if (threadIdx.x == 0) {
            shared[2] = 0;
            claim = atomicAdd(a.ticket, 1);
        }
    }
    // A wait ran out (any thread): the next unit is none, so that the block ends instead of waiting again for each.
    __device__ void stop() { shared[2] = 1; }
    // The next unit (total or more: none is left), and the set that this block has to join, or -1. All threads; the
    // barriers also free the unit's shared memory.
    __device__ int next(int& join) {
        if (threadIdx.x == 0) {
            shared[0] = claim;
            shared[1] = set >= 0 && count == a.p.units - 1 ? set : -1;
        }
        __syncthreads();
        const int t = shared[2] ? total : shared[0];
        join = shared[1];
        set = -1;
        __syncthreads();
        if (threadIdx.x == 0 && t < total) claim = atomicAdd(a.ticket, 1);
        return t;
    }
    // The unit's sums are written (by all threads).
    __device__ void summed(int of) {
        __syncthreads();
        set = of;
        if (threadIdx.x == 0) {
            __threadfence();
            count = atomicAdd(a.done + of, 1);
        }
    }
};

// The set's sums are joined (written by all threads): its second pass may go.
__device__ __forceinline__ void release_set(const Args& a, int set) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicExch(a.ready + set, 1);
    }
}

// Waits, a warp by itself, until the set's sums are joined; false when the bounded wait ran out.
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

// ---------------------------------------------------------------- forward --

// Joins a set's units: mean and rstd of its groups.
__device__ __forceinline__ void join_stats(const Args& a, int set, float* stats) {
    const NormShape& s = a.s;
    const Plan& p = a.p;
    const int cg = s.C / s.groups, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Place c = place_of(a, set, 0);
    const float total = (float)s.HW * (float)cg;
    __threadfence();
    for (int g = warp; g < c.ng; g += NT / 32) {
        const float2* first = a.pieces + ((size_t)c.b * p.chunks * s.groups + c.g0 + g) * p.parts;
        auto piece = [&](int i) { return ld_l2(first + (size_t)(i / p.parts) * s.groups * p.parts + i % p.parts); };
        auto count = [&](int i) {
            const int ch = i / p.parts, pt = i % p.parts;
            const int w = p.gpb ? cg : min(p.cb, cg - pt * p.cb);
            return (float)(min((ch + 1) * p.rows, s.HW) - ch * p.rows) * (float)w;
        };
        float u = 0.f;
#pragma unroll 4
        for (int i = lane; i < p.units; i += 32) u += piece(i).x * (count(i) / total);
        const float mean = warp_sum(u);
        float m2 = 0.f;
#pragma unroll 4
        for (int i = lane; i < p.units; i += 32) {
            const float2 q = piece(i);
            m2 += q.y + count(i) * (q.x - mean) * (q.x - mean);
        }
        m2 = warp_sum(m2);
        if (lane == 0) {
            const float2 v = make_float2(mean, rsqrtf(m2 / total + s.eps));
            const size_t o = (size_t)c.b * s.groups + c.g0 + g;
            a.sets[o] = v;
            if (stats) {
                stats[2 * o] = v.x;
                stats[2 * o + 1] = v.y;
            }
        }
    }
    release_set(a, set);
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(NT, 3)
    forward_kernel(const Args a, const T* __restrict__ x, const T* __restrict__ gamma, const T* __restrict__ beta,
                   T* __restrict__ y, float* __restrict__ stats) {
    __shared__ float sm[2 * NT * V];  // [2][ty][cb] sums, reused as [2][cb]
    __shared__ int shared[3];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const NormShape& s = a.s;
    const Plan& p = a.p;
    const int cg = s.C / s.groups, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int tx = (p.cb + V - 1) / V, ty = NT / tx, cx = threadIdx.x % tx, ry = threadIdx.x / tx;
    Queue queue(a, shared);
    int params_at = -1;  // the channels whose gamma and beta are held
    float ga[V], be[V];
    for (;;) {
        int join;
        const int t = queue.next(join);
        if (join >= 0) join_stats(a, join, stats);
        if (t >= queue.total) break;
        int pass, set, unit;
        unit_at(a, t, pass, set, unit);
        const Place c = place_of(a, set, unit);
        const bool in = ry < ty && cx * V < c.nc;
        const size_t at = (size_t)c.b * s.HW * s.C + c.c0 + cx * V;
        const T* xp = x + at;
        if (pass == 0) {
            const int rows = c.r1 - c.r0;
            if (in) {
                // see Running: k the level, s1 and s2 the sums about it
                float k[V], s1[V] = {}, s2[V] = {};
                int n = 0, next = 8;
                load<T, V>(k, xp + (size_t)min(c.r0 + ry, c.r1 - 1) * s.C);
                auto add = [&](const float(&v)[V]) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float d = v[i] - k[i];
                        s1[i] += d;
                        s2[i] = fmaf(d, d, s2[i]);
                    }
                };
                auto level = [&]() {
                    const float inv = n > 0 ? 1.f / (float)n : 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float m = s1[i] * inv;
                        s2[i] = fmaf(-s1[i], m, s2[i]);
                        k[i] += m;
                        s1[i] = 0.f;
                    }
                };
                int r = c.r0 + ry;
                for (; r + 7 * ty < c.r1; r += 8 * ty) {
                    typename std::conditional<V == 1, float, uint4>::type q[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const T* at = xp + (size_t)(r + j * ty) * s.C;
                        if constexpr (V > 1) q[j] = ptx::ldg_v4_stream(at);
                        else q[j] = ld1(at);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float v[V];
                        if constexpr (V > 1) unpack(v, q[j]);
                        else v[0] = q[j];
                        add(v);
                    }
                    n += 8;
                    if (n == next) {
                        level();
                        next *= 2;
                    }
                }
#pragma unroll 4
                for (; r < c.r1; r += ty, ++n) {
                    float v[V];
                    load<T, V>(v, xp + (size_t)r * s.C);
                    add(v);
                }
                level();
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    sm[ry * p.cb + cx * V + i] = k[i];
                    sm[(ty + ry) * p.cb + cx * V + i] = s2[i];
                }
            }
            __syncthreads();
            const float n = (float)rows;
            const int each = rows / ty, more = rows % ty;
            for (int q = threadIdx.x; q < c.nc; q += NT)
                join_slots(sm + q, p.cb, ty, n, [&](int r) { return (float)(each + (r < more)); });
            __syncthreads();
            // a warp joins the channels of a group: all have n values
            const int cw = p.gpb ? cg : c.nc;
            for (int g = warp; g < c.ng; g += NT / 32) {
                float u = 0.f;
                for (int q = lane; q < cw; q += 32) u += sm[g * cw + q];
                const float mean = warp_sum(u) / (float)cw;
                float m2 = 0.f;
                for (int q = lane; q < cw; q += 32) {
                    const float d = sm[g * cw + q] - mean;
                    m2 += sm[ty * p.cb + g * cw + q] + n * d * d;
                }
                m2 = warp_sum(m2);
                if (lane == 0)
                    a.pieces[(((size_t)c.b * p.chunks + c.chunk) * s.groups + c.g0 + g) * p.parts + c.part] =
                        make_float2(mean, m2);
            }
            queue.summed(set);
        } else {
            if (params_at != c.c0) {
                params_at = c.c0;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    ga[i] = gamma && in ? ld1(gamma + c.c0 + cx * V + i) : 1.f;
                    be[i] = beta && in ? ld1(beta + c.c0 + cx * V + i) : 0.f;
                }
            }
            // the first pixels are on their way while the set's statistics are waited for
            uint4 q[8];
            int r = c.r0 + ry;
            bool ahead = false;
            if constexpr (V > 1) {
                ahead = in && r + 7 * ty < c.r1;
                if (ahead)
#pragma unroll
                    for (int j = 0; j < 8; ++j) q[j] = ptx::ldg_v4_stream(xp + (size_t)(r + j * ty) * s.C);
            }
            if (!await_set(a, set)) {
                queue.stop();
                continue;
            }
            if (!in) continue;
            float m[V], sc[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 v = ld_l2(a.sets + (size_t)c.b * s.groups + (c.c0 + cx * V + i) / cg);
                m[i] = v.x;
                sc[i] = v.y * ga[i];
            }
            T* yp = y + at;
            if constexpr (V > 1) {
                while (ahead) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float v[V];
                        unpack(v, q[j]);
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            v[i] = act_apply<ACT, kFast<T>>(fmaf(v[i] - m[i], sc[i], be[i]));
                        store<T, V>(yp + (size_t)(r + j * ty) * s.C, v);
                    }
                    r += 8 * ty;
                    ahead = r + 7 * ty < c.r1;
                    if (ahead)
#pragma unroll
                        for (int j = 0; j < 8; ++j) q[j] = ptx::ldg_v4_stream(xp + (size_t)(r + j * ty) * s.C);
                }
            }
#pragma unroll 4
            for (; r < c.r1; r += ty) {
                float v[V];
                load<T, V>(v, xp + (size_t)r * s.C);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = act_apply<ACT, kFast<T>>(fmaf(v[i] - m[i], sc[i], be[i]));
                store<T, V>(yp + (size_t)r * s.C, v);
            }
        }
    }
}

// --------------------------------------------------------------- backward --

// Joins a set's units: the sums of its channels, c1 and c2 of its groups; the last set of all, the parameters'
// gradients.
template <typename T>
__device__ __forceinline__ void join_sums(const Args& a, int set, const T* gamma, float* gg, float* gb, int* flag) {
    const NormShape& s = a.s;
    const Plan& p = a.p;
    const int cg = s.C / s.groups, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Place c = place_of(a, set, 0);
    float2* csums = a.sets;
    float2* c12 = a.sets + (size_t)s.B * s.C;
    const int c0 = c.g0 * cg, nc = c.ng * cg;  // (parts) the whole group
    __threadfence();
    for (int q = c0 + threadIdx.x; q < c0 + nc; q += NT) {
        float2 v = make_float2(0.f, 0.f);
#pragma unroll 8
        for (int i = 0; i < p.chunks; ++i) {
            const float2 w = ld_l2(a.pieces + ((size_t)c.b * p.chunks + i) * s.C + q);
            v.x += w.x;
            v.y += w.y;
        }
        csums[(size_t)c.b * s.C + q] = v;
    }
    __syncthreads();
    const float inv = 1.f / ((float)s.HW * (float)cg);
    for (int g = c.g0 + warp; g < c.g0 + c.ng; g += NT / 32) {
        float u = 0.f, d = 0.f;
        for (int q = g * cg + lane; q < (g + 1) * cg; q += 32) {
            const float2 w = ld_l2(csums + (size_t)c.b * s.C + q);
            const float k = gamma ? ld1(gamma + q) : 1.f;
            u = fmaf(k, w.x, u);
            d = fmaf(k, w.y, d);
        }
        u = warp_sum(u);
        d = warp_sum(d);
        if (lane == 0) c12[(size_t)c.b * s.groups + g] = make_float2(u * inv, d * inv);
    }
    release_set(a, set);
    if (gg || gb) {
        if (threadIdx.x == 0) *flag = atomicAdd(a.finished, 1) == s.B * p.sets - 1;
        __syncthreads();
        if (*flag) {
            __threadfence();
            for (int q = threadIdx.x; q < s.C; q += NT) params_of(s, csums, q, gg, gb);
        }
    }
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(NT, 2)
    backward_kernel(const Args a, const T* __restrict__ x, const T* __restrict__ gamma, const T* __restrict__ beta,
                    const float* __restrict__ stats, const T* __restrict__ gy, T* __restrict__ gx,
                    float* __restrict__ gg, float* __restrict__ gb) {
    __shared__ float sm[2 * NT * V];  // [2][ty][cb]
    __shared__ int shared[3], flag;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const NormShape& s = a.s;
    const Plan& p = a.p;
    const int cg = s.C / s.groups;
    const int tx = (p.cb + V - 1) / V, ty = NT / tx, cx = threadIdx.x % tx, ry = threadIdx.x / tx;
    const float2* c12 = a.sets + (size_t)s.B * s.C;  // [B][groups] (c1, c2)
    Queue queue(a, shared);
    int params_at = -1;  // the channels whose gamma and beta are held
    float ga[V], be[V];
    for (;;) {
        int join;
        const int t = queue.next(join);
        if (join >= 0) join_sums(a, join, gamma, gg, gb, &flag);
        if (t >= queue.total) break;
        int pass, set, unit;
        unit_at(a, t, pass, set, unit);
        if (pass == 1 && !gx) continue;
        const Place c = place_of(a, set, unit);
        const bool in = ry < ty && cx * V < c.nc;
        const size_t at = (size_t)c.b * s.HW * s.C + c.c0 + cx * V;
        if (params_at != c.c0) {
            params_at = c.c0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                ga[i] = gamma && in ? ld1(gamma + c.c0 + cx * V + i) : 1.f;
                be[i] = beta && in ? ld1(beta + c.c0 + cx * V + i) : 0.f;
            }
        }
        // the first pixels are on their way while the statistics are read and (second pass) waited for
        uint4 q[4], h[4];
        int r = c.r0 + ry;
        auto fetch = [&]() {
            if constexpr (V > 1) {
                const bool go = in && r + 3 * ty < c.r1;
                if (go) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) q[j] = ptx::ldg_v4_stream(x + at + (size_t)(r + j * ty) * s.C);
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[j] = ptx::ldg_v4_stream(gy + at + (size_t)(r + j * ty) * s.C);
                }
                return go;
            }
            return false;
        };
        bool ahead = fetch();
        float mean[V], rstd[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float* st = stats + ((size_t)c.b * s.groups + min(c.c0 + cx * V + i, s.C - 1) / cg) * 2;
            mean[i] = __ldg(st);
            rstd[i] = __ldg(st + 1);
        }
        // f(r, dz values, xh values) for each of the thread's pixels, after(n) behind n of them
        auto walk = [&](auto&& f, auto&& after) {
            auto one = [&](int row, const float(&v)[V], const float(&g)[V]) {
                float d[V], hat[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    hat[i] = (v[i] - mean[i]) * rstd[i];
                    d[i] = dz_of<ACT, kFast<T>>(g[i], v[i], hat[i], mean[i], rstd[i], ga[i], be[i]);
                }
                f(row, d, hat);
            };
            if constexpr (V > 1) {
                while (ahead) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float v[V], g[V];
                        unpack(v, q[j]);
                        unpack(g, h[j]);
                        one(r + j * ty, v, g);
                    }
                    after(4);
                    r += 4 * ty;
                    ahead = fetch();
                }
            }
#pragma unroll 2
            for (; r < c.r1; r += ty) {
                float v[V], g[V];
                load<T, V>(v, x + at + (size_t)r * s.C);
                load<T, V>(g, gy + at + (size_t)r * s.C);
                one(r, v, g);
                after(1);
            }
        };
        if (pass == 0) {
            if (in) {
                // sums of kRun pixels, and sums of those: no chain grows with the map
                float s1[V] = {}, s2[V] = {}, t1[V] = {}, t2[V] = {};
                int run = 0;
                auto close = [&]() {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        t1[i] += s1[i];
                        t2[i] += s2[i];
                        s1[i] = s2[i] = 0.f;
                    }
                    run = 0;
                };
                walk(
                    [&](int, const float(&d)[V], const float(&hat)[V]) {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            s1[i] += d[i];
                            s2[i] = fmaf(d[i], hat[i], s2[i]);
                        }
                    },
                    [&](int n) {
                        if ((run += n) >= kRun) close();
                    });
                close();
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    sm[ry * p.cb + cx * V + i] = t1[i];
                    sm[(ty + ry) * p.cb + cx * V + i] = t2[i];
                }
            }
            __syncthreads();
            for (int k = threadIdx.x; k < c.nc; k += NT) {
                float u = 0.f, d = 0.f;
#pragma unroll 8
                for (int row = 0; row < ty; ++row) {
                    u += sm[row * p.cb + k];
                    d += sm[(ty + row) * p.cb + k];
                }
                a.pieces[((size_t)c.b * p.chunks + c.chunk) * s.C + c.c0 + k] = make_float2(u, d);
            }
            queue.summed(set);
        } else {
            if (!await_set(a, set)) {
                queue.stop();
                continue;
            }
            if (!in) continue;
            float c1[V], c2[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 v = ld_l2(c12 + (size_t)c.b * s.groups + (c.c0 + cx * V + i) / cg);
                c1[i] = v.x;
                c2[i] = v.y;
            }
            walk([&](int row, const float(&d)[V], const float(&hat)[V]) {
                float v[V];
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = rstd[i] * (fmaf(ga[i], d[i], -c1[i]) - hat[i] * c2[i]);
                store<T, V>(gx + at + (size_t)row * s.C, v);
            }, [](int) {});
        }
    }
}

// The parameters' gradients alone, from a sample's sums [B][C]. 32 channels a block, a warp a row of them; the warps of a
// cluster's blocks share the samples. Each adds runs of 32 and the runs in float64, so that no float32 chain grows with
// the samples (in one thread a channel, 4096 equal samples were off by 800 of 2^-24), and all are joined in a fixed
// order. The whole backward of 4096x7x7x256 took 639 us with one thread a channel, 221 so; of 8x50x50x256 17.5 either way.
constexpr int PARAMS_WARPS = 8, PARAMS_CLUSTER = 8, PARAMS_RUN = 32;

__global__ void __launch_bounds__(PARAMS_WARPS * 32)
    params_kernel(const NormShape s, const float2* __restrict__ sums, float* gg, float* gb, int ctas) {
    __shared__ float part[2][PARAMS_WARPS][32], joined[2][32];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, rank = blockIdx.x % ctas;
    const int c = blockIdx.x / ctas * 32 + lane, step = ctas * PARAMS_WARPS;
    double u = 0.0, d = 0.0;
    if (c < s.C)
        for (long long b0 = rank * PARAMS_WARPS + warp; b0 < s.B; b0 += (long long)PARAMS_RUN * step) {
            float2 run = make_float2(0.f, 0.f);
#pragma unroll 8
            for (int k = 0; k < PARAMS_RUN; ++k) {
                const long long b = b0 + (long long)k * step;
                if (b >= s.B) break;
                const float2 q = __ldcg(sums + b * s.C + c);
                run.x += q.x;
                run.y += q.y;
            }
            u += run.x;
            d += run.y;
        }
    part[0][warp][lane] = (float)u;
    part[1][warp][lane] = (float)d;
    __syncthreads();
    if (warp < 2) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < PARAMS_WARPS; ++w) v += part[warp][w][lane];
        joined[warp][lane] = v;
    }
    if (ctas > 1) {
        ptx::cluster_sync();
        if (warp < 2 && rank == 0) {
            float v = 0.f;
            for (int k = 0; k < ctas; ++k) v += ld_cluster(ptx::smem_u32(&joined[warp][lane]), k);
            joined[warp][lane] = v;
        }
        ptx::cluster_sync();  // no block leaves before it has been read
    }
    float* out = warp == 0 ? gb : gg;
    if (warp < 2 && rank == 0 && c < s.C && out) out[c] = joined[warp][lane];
}

// ------------------------------------------------------------------- host --

template <typename F, typename... Q>
cudaError_t launch(F f, int grid, int threads, cudaStream_t st, Q... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, f, args...);
}

cudaError_t params_of_samples(const NormShape& s, const float2* sums, float* gg, float* gb, cudaStream_t st,
                              int* launches) {
    const int ctas = s.B > 8 * PARAMS_WARPS ? PARAMS_CLUSTER : 1;  // one batch of loads a thread needs no cluster
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((s.C + 31) / 32 * ctas));
    cfg.blockDim = dim3(PARAMS_WARPS * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    ++*launches;
    return cudaLaunchKernelEx(&cfg, params_kernel, s, sums, gg, gb, ctas);
}

cudaError_t args_of(const NormShape& s, const Plan& p, bool backward, void* ws, unsigned* status, cudaStream_t st,
                    Args& a, int* launches) {
    const Space w = space_of(s, p, backward);
    uint8_t* base = static_cast<uint8_t*>(ws);
    int* counters = reinterpret_cast<int*>(base + w.counters);
    a.s = s;
    a.p = p;
    a.ticket = counters;
    a.finished = counters + 1;
    a.done = counters + 2;
    a.ready = a.done + (size_t)s.B * p.sets;
    a.pieces = reinterpret_cast<float2*>(base + w.pieces);
    a.sets = reinterpret_cast<float2*>(base + w.sets);
    a.status = status;
    ++*launches;
    return cudaMemsetAsync(counters, 0, (2 + 2 * (size_t)s.B * p.sets) * sizeof(int), st);
}

template <typename T, int V>
cudaError_t forward_v(const Args& a, const T* x, const T* gamma, const T* beta, T* y, float* stats, cudaStream_t st) {
    return with_act(a.s.act, [&](auto A) {
        return launch(forward_kernel<T, V, decltype(A)::value>, a.p.grid, NT, st, a, x, gamma, beta, y, stats);
    });
}

template <typename T, int V>
cudaError_t backward_v(const Args& a, const T* x, const T* gamma, const T* beta, const float* stats, const T* gy, T* gx,
                       float* gg, float* gb, cudaStream_t st) {
    return with_act(a.s.act, [&](auto A) {
        return launch(backward_kernel<T, V, decltype(A)::value>, a.p.grid, NT, st, a, x, gamma, beta, stats, gy, gx, gg,
                      gb);
    });
}

template <typename T>
constexpr int vec_of() {
    return 16 / (int)sizeof(T);
}

template <typename T>
cudaError_t forward_t(const NormShape& s, bool vec, const T* x, const T* gamma, const T* beta, T* y, float* stats,
                      void* ws, unsigned* status, cudaStream_t st, int* launches) {
    constexpr int V = vec_of<T>();
    const Plan p = make_plan(s, vec ? V : s.C + 1, sizeof(T), 1);
    Args a;
    const cudaError_t e = args_of(s, p, false, ws, status, st, a, launches);
    if (e != cudaSuccess) return e;
    ++*launches;
    return p.V == V ? forward_v<T, V>(a, x, gamma, beta, y, stats, st) : forward_v<T, 1>(a, x, gamma, beta, y, stats, st);
}

template <typename T>
cudaError_t backward_t(const NormShape& s, bool vec, const T* x, const T* gamma, const T* beta, const float* stats,
                       const T* gy, T* gx, float* gg, float* gb, void* ws, unsigned* status, cudaStream_t st,
                       int* launches) {
    constexpr int V = vec_of<T>();
    const Plan p = make_plan(s, vec ? V : s.C + 1, sizeof(T), 2);
    Args a;
    cudaError_t e = args_of(s, p, true, ws, status, st, a, launches);
    if (e != cudaSuccess) return e;
    ++*launches;
    const bool apart = s.B > kFewSamples && (gg || gb);
    float *g1 = apart ? nullptr : gg, *g2 = apart ? nullptr : gb;
    e = p.V == V ? backward_v<T, V>(a, x, gamma, beta, stats, gy, gx, g1, g2, st)
                 : backward_v<T, 1>(a, x, gamma, beta, stats, gy, gx, g1, g2, st);
    return e == cudaSuccess && apart ? params_of_samples(s, a.sets, gg, gb, st, launches) : e;
}

}  // namespace

namespace {

// Which kernels an aligned map goes to. Clusters need one launch; the queue with a ring, two, moves large maps faster:
// relu on 8x50x50x256 11.5 and 18.5 us, on 8x80x80x256 (26 MB) 28.2 and 27.5 us, on 64x28x28x512 51 and 37 us, on
// 4096x7x7x256 197 and 161.
// (Backward the clusters lead wherever they fit: 64x28x28x512 82 and 118 us.)
enum class Path { cluster, stream, queue };
Path path_of(const NormShape& s, int bf, bool backward) {
    const bool stream = norm_stream_supported(s, bf, backward);
    const bool large = !backward && (double)s.B * s.HW * s.C * (bf ? 2 : 4) > 24e6 && stream;
    if (!large && norm_cluster_supported(s, bf, backward)) return Path::cluster;
    return stream ? Path::stream : Path::queue;
}

size_t queue_workspace(const NormShape& s, int bf, bool backward, int vec) {
    return space_of(s, make_plan(s, vec, bf ? 2 : 4, backward ? 2 : 1), backward).total;
}

}  // namespace

size_t norm_workspace(const NormShape& s, int bf, bool backward, bool aligned) {
    size_t n = 0;
    switch (path_of(s, bf, backward)) {
        case Path::cluster: n = backward ? (size_t)s.B * s.C * sizeof(float2) : 0; break;
        case Path::stream: n = norm_stream_workspace(s, bf, backward); break;
        case Path::queue: n = queue_workspace(s, bf, backward, bf ? 8 : 4); break;
    }
    return aligned ? n : std::max(n, queue_workspace(s, bf, backward, s.C + 1));  // C + 1: single values
}

cudaError_t norm_forward(const NormShape& s, int bf, bool vec, const void* x, const void* gamma, const void* beta,
                         void* y, float* stats, void* ws, unsigned* status, cudaStream_t st, int* launches) {
    const Path path = vec ? path_of(s, bf, false) : Path::queue;
    if (path == Path::cluster) {
        ++*launches;
        return norm_cluster_forward(s, bf, x, gamma, beta, y, stats, st);
    }
    if (path == Path::stream) {
        *launches += 2;
        return norm_stream_forward(s, bf, x, gamma, beta, y, stats, ws, status, st);
    }
    return bf ? forward_t(s, vec, (const bf16*)x, (const bf16*)gamma, (const bf16*)beta, (bf16*)y, stats, ws, status,
                          st, launches)
              : forward_t(s, vec, (const float*)x, (const float*)gamma, (const float*)beta, (float*)y, stats, ws,
                          status, st, launches);
}

cudaError_t norm_backward(const NormShape& s, int bf, bool vec, const void* x, const void* gamma, const void* beta,
                          const float* stats, const void* gy, void* gx, float* gg, float* gb, void* ws,
                          unsigned* status, cudaStream_t st, int* launches) {
    const Path path = vec ? path_of(s, bf, true) : Path::queue;
    if (path == Path::cluster) {
        float2* sums = gg || gb ? (float2*)ws : nullptr;
        const cudaError_t e = norm_cluster_backward(s, bf, x, gamma, beta, stats, gy, sums, gx, st);
        if (e != cudaSuccess) return e;
        ++*launches;
        return sums ? params_of_samples(s, sums, gg, gb, st, launches) : e;
    }
    if (path == Path::stream) {
        *launches += 2;
        const bool apart = s.B > kFewSamples && (gg || gb);
        const cudaError_t e = norm_stream_backward(s, bf, x, gamma, beta, stats, gy, gx, apart ? nullptr : gg,
                                                   apart ? nullptr : gb, ws, status, st);
        if (e != cudaSuccess || !apart) return e;
        return params_of_samples(s, norm_stream_sums(s, bf, ws), gg, gb, st, launches);
    }
    return bf ? backward_t(s, vec, (const bf16*)x, (const bf16*)gamma, (const bf16*)beta, stats, (const bf16*)gy,
                           (bf16*)gx, gg, gb, ws, status, st, launches)
              : backward_t(s, vec, (const float*)x, (const float*)gamma, (const float*)beta, stats, (const float*)gy,
                           (float*)gx, gg, gb, ws, status, st, launches);
}

}  // namespace dcn
