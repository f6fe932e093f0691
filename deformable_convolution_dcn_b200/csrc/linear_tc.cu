// The linear layer's matrix products on sm_100a tensor cores:
//   forward      D[m, n] = sum_k x[m, k] W[n, k]      both operands K-major
//   grad_x       D[m, k] = sum_n dz[m, n] W[n, k]     W MN-major
//   grad_weight  D[n, k] = sum_m dz[m, n] x[m, k]     both MN-major
// One persistent kernel computes them all, D = A B^T with A's rows on the TMEM
// lanes (128 a CTA) and BN of B's rows on its columns. Either matrix may take
// A's place; D is then written transposed (products of few rows put the long
// side on the lanes). CG = 2 runs two CTAs as one tile of 256 rows (cta_group::2),
// each holding half of B's rows, which halves the L2 traffic of B.
//
// float32 accuracy from bfloat16 products: a float32 operand is split beforehand
// in three bfloat16 terms a0 + a1 + a2 (24 bits), and the product is
// a0 b0 + (a0 b1 + a1 b0 + a1 b1 + a0 b2 + a2 b0); the terms left out are below
// 2^-26 of a b. a0 b0 has an accumulator of its own, so that the small products
// do not make it round more often, and stands alone where it is infinite or NaN:
// an infinity has zeros for its other terms, whose products would make it NaN. The tensor cores cut each step's sum off
// rather than rounding it, so float32 results take the accumulator out every
// `chunk` blocks of 64 and add it in registers with proper rounding. bfloat16
// results, whose rounding is off by up to 2e-3, do so where the reduction is over 64
// blocks, in equal pieces of up to 64: left whole, 12544 positive products lost 5.8e-5
// of their sum, 65536 lost 1.6e-4, 401408 lost 8.6e-4; in pieces they lose 4e-6 at any
// length (4000x1024x12544 75.4 us, whole 73.7).
//
// Warps: 0 and 10 TMA producers of A and B, 1 MMA issue and TMEM, 2-9 epilogue
// (each of the four TMEM lane quarters twice, once for each half of the columns). Accumulators
// are double buffered: the epilogue of a tile overlaps the next one's MMAs. The
// epilogue adds bias and residual, applies the activation and stores whole
// 32-byte sectors. Products with too few tiles to fill the GPU are split along
// the reduction; the parts meet in finish_kernel, in a fixed order.
//
// Measured (M x N x K, GPU time): bfloat16 4000x1024x12544 relu 75 us, 1363 TFLOP/s,
// the tensor pipe busy 86 % of the cycles, backward 180; 20000x1024x256 18 us, bound by
// the result's bytes (14.4 where L2 holds x), and 25.5 with relu and a shortcut; backward
// 20000x256x1024 relu 53 us, 5000x2048x512 gelu 87 us, of which the preparation of dz takes
// 13 to 18; float32 8192x2048x2048 293 to 310 us, 1350 TFLOP/s of bfloat16 products
// (power-bound).
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "act.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace dcn {
namespace {

constexpr int BM = 128, BK = 64;          // lanes a CTA, reduction elements a stage
constexpr int EPI_WARPS = 8;
constexpr int B_WARP = 2 + EPI_WARPS;     // the second producer
constexpr int THREADS = (B_WARP + 1) * 32;
constexpr int MAX_STAGES = 8;
constexpr uint32_t A_BYTES = BM * BK * 2; // one term of one stage
constexpr uint32_t MN_BLOCK = BK * 128;   // 64 rows of an MN-major operand over a stage: 8 KB
constexpr int MAX_SLOTS = 3;
constexpr uint32_t SMEM_MAX = 227 * 1024, BAR_BYTES = 512;
constexpr uint32_t SLOT_BYTES = 4096, EXCHANGE_BYTES = 32 * 33 * 4, BIAS_BYTES = 128 * 4;  // a warp
constexpr uint32_t TMEM_COLS = 512;
constexpr int LONG = 64;                  // stages that a bfloat16 result's accumulator adds up at most
constexpr long long WAIT_LIMIT = 2000000000LL;

// How the TMA producer walks an operand (see encode()).
constexpr int kKMajor = 0, kMnBlocks = 1, kMnRows = 2;
struct Operand {
    int terms;  // bfloat16 terms: 1 or 3 (one side of a bfloat16 result: or 2)
    int kind;
};

// grad_bias from the column sums of row blocks (gb null: not asked for).
struct Sums {
    const float* sums;
    int blocks, pitch, n;
    float* gb;
};
struct GemmArgs {
    int rows, cols;        // D: A-side rows, B-side rows
    int kblocks, splits;   // stages of 64; parts along the reduction
    int kper, kmore;       // stages a part, and parts with one more
    int chunk;             // stages between two reads of the accumulator
    int mt, nt;            // tiles
    int bn;                // B rows a tile (of the CTA or pair)
    Operand a, b;
    int stages;
    uint32_t stage_bytes, bar_off;
    // epilogue: D[i, j] goes to element i * rs + j * cs
    long long rs, cs, part;  // part: elements between two splits' results
    const void *bias, *residual;
    void *y, *z;
    int act;
    int one_column;        // the result has one, and one bias: swapped, D is walked as if it were not (cs = 1)
    int tma_out;           // D's rows are 16-byte aligned and written as they lie: TMA stores
    int nslots;            // chunks a warp stages (tma_out)
    uint32_t slot_off, sm_off;  // the epilogue's slots or exchange buffers; its bias
    unsigned* status;
    Sums gb;               // grad_bias, joined by the epilogue warps while they wait for the first accumulator
};

// Shared-memory descriptors of one operand's tiles. Only the start address (the low word, in 16-byte units) changes
// from one MMA to the next: by `step` for 16 reduction elements (K-major: 32 bytes on; MN-major: 16 rows of 128
// bytes on, with blocks of 64 rows MN_BLOCK apart as leading byte offset).
struct OperandDesc {
    uint32_t low, high, step;
    __device__ OperandDesc(uint32_t addr, int mn) {
        uint64_t d = ptx::sw128_desc(addr);
        if (mn) d = (d & ~((uint64_t)0x3FFFu << 16)) | ((uint64_t)(MN_BLOCK >> 4) << 16);
        low = (uint32_t)d;
        high = (uint32_t)(d >> 32);
        step = mn ? 2048 / 16 : 32 / 16;
    }
    // k: steps, off: 16-byte units (no carry leaves the address field: shared memory ends below 2^18)
    __device__ __forceinline__ uint64_t at(uint32_t off, int k) const {
        return ((uint64_t)high << 32) | (low + off + k * step);
    }
};

template <bool FAST>
__device__ __forceinline__ float act_run(float z, int act) {
    switch (act) {
        case kActRelu: return act_apply<kActRelu, FAST>(z);
        case kActSilu: return act_apply<kActSilu, FAST>(z);
        case kActGelu: return act_apply<kActGelu, FAST>(z);
        default: return z;
    }
}

template <int ACT, bool FAST>
__device__ __forceinline__ void act32(float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = act_apply<ACT, FAST>(v[i]);
}

// 16 bytes of a row of D: 8 bfloat16 or 4 float32 values.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* v) {
    if constexpr (std::is_same<T, float>::value) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    } else {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        return *reinterpret_cast<uint4*>(h);
    }
}
template <typename T>
__device__ __forceinline__ void add16(float* v, uint4 w) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, float>::value) {
            v[i] += __uint_as_float(q[i]);
        } else {
            v[2 * i] += __uint_as_float(q[i] << 16);
            v[2 * i + 1] += __uint_as_float(q[i] & 0xFFFF0000u);
        }
    }
}

// One warp's epilogue: 32 rows of D, one a lane, in chunks of 128 bytes a row. A chunk goes out through a 4 KB
// shared-memory slot of the warp by a TMA store of its own (a lane writes 16-byte pieces of its row, 128-byte
// swizzled: no bank conflicts, where direct stores would touch 32 lines an instruction), and the residual comes in
// by TMA through the slots ahead, to be overwritten in place; no two warps wait for each other.
template <typename T>
struct Emit {
    static constexpr int COLS = 128 / (int)sizeof(T);  // columns a chunk
    const GemmArgs& a;
    const CUtensorMap *my, *mz, *mr;
    T *y, *z;
    const T *bias, *residual;
    uint32_t slots, resbar;  // shared addresses of the warp's slots and of their residual barriers
    float *sm, *sbias;       // exchange buffer (32 x 33), bias of the warp's columns
    volatile int* abort;
    int lane;
    // the chunk's place
    int row0, sp;
    int out = 0;             // chunks written
    int in = 0;              // residual chunks asked for
    bool ok = true;

    __device__ __forceinline__ bool active(int row, int col) const { return row < a.rows && col < a.cols; }
    // the residual of one active chunk into its slot (the slot's last store has been read)
    __device__ __forceinline__ void fetch(int row, int col) {
        if (lane == 0) {
            const int s = in % a.nslots;
            ptx::mbar_arrive_expect_tx(resbar + s * 8, 4096);
            ptx::tma_load_3d(slots + s * 4096, mr, resbar + s * 8, col, row, 0);
        }
        ++in;
    }
    // `v`: COLS columns from `col`, whose bias is sbias[b..]
    __device__ __forceinline__ void chunk(float (&v)[COLS], int col, int b, bool epilogue) {
        if (!a.tma_out) {
            if (active(row0, col))
#pragma unroll
                for (int i = 0; i < COLS; i += 32)
                    through_shared(*reinterpret_cast<float(*)[32]>(&v[i]), col + i);
            return;
        }
        if (!active(row0, col)) return;
        const int s = out % a.nslots;
        const uint32_t slot = slots + s * 4096, mine = slot + lane * 128;
        if (epilogue) {
            if (bias) {
#pragma unroll
                for (int i = 0; i < COLS; i += 4) {
                    const float4 w = *reinterpret_cast<const float4*>(sbias + b + i);
                    v[i] += w.x, v[i + 1] += w.y, v[i + 2] += w.z, v[i + 3] += w.w;
                }
            }
            if (residual) {
                ok = ptx::mbar_wait(resbar + s * 8, (out / a.nslots) & 1, abort, a.status, WAIT_LIMIT) && ok;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    add16<T>(&v[i * kVec<T>], ptx::lds_v4(mine + ((i ^ (lane & 7)) << 4)));
            }
        }
        // a slot is written again once the store before has read it (lane 0 issued it)
        if (!residual && lane == 0) {
            if (a.nslots == 2) ptx::bulk_wait_group_read<1>();
            else ptx::bulk_wait_group_read<0>();
        }
        __syncwarp();
        if (epilogue && z) {
            put(v, mine);
            send(mz, slot, col);
            if (lane == 0) ptx::bulk_wait_group_read<0>();
            __syncwarp();
        }
        if (epilogue) {
            switch (a.act) {
                case kActRelu: act_all<kActRelu>(v); break;
                case kActSilu: act_all<kActSilu>(v); break;
                case kActGelu: act_all<kActGelu>(v); break;
                default: break;
            }
        }
        put(v, mine);
        send(my, slot, col);
        ++out;
    }
    // the slot of the chunk before has been read by its store: a residual chunk may be fetched into it
    __device__ __forceinline__ void freed() {
        if (lane == 0) ptx::bulk_wait_group_read<1>();
        __syncwarp();
    }
    template <int ACT>
    __device__ __forceinline__ void act_all(float (&v)[COLS]) {
#pragma unroll
        for (int i = 0; i < COLS; ++i) v[i] = act_apply<ACT, kFast<T>>(v[i]);
    }
    __device__ __forceinline__ void put(const float (&v)[COLS], uint32_t mine) {
#pragma unroll
        for (int i = 0; i < 8; ++i) ptx::sts_v4(mine + ((i ^ (lane & 7)) << 4), pack16<T>(&v[i * kVec<T>]));
    }
    __device__ __forceinline__ void send(const CUtensorMap* m, uint32_t slot, int col) {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            ptx::tma_store_3d(m, slot, col, row0, sp);
            ptx::bulk_commit_group();
        }
    }
    // Rows that are not whole vectors, and D written transposed: the values change lanes in shared memory, so that a
    // warp's accesses lie side by side either way.
    __device__ __forceinline__ void through_shared(const float (&v)[32], int col) {
        if (col >= a.cols) return;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) sm[lane * 33 + i] = v[i];
        __syncwarp();
        const bool rows_on_lanes = a.cs != 1;
        const int mine = (rows_on_lanes ? row0 : col) + lane;  // this lane's row or column
        const int n = min(32, rows_on_lanes ? a.cols - col : a.rows - row0);
        if (mine < (rows_on_lanes ? a.rows : a.cols)) {
            const float b = bias ? ld1(bias + (a.one_column ? 0 : mine)) : 0.f;
            long long at = rows_on_lanes ? mine + col * a.cs : row0 * a.rs + mine;
            const long long step = rows_on_lanes ? a.cs : a.rs;
            const float* p = rows_on_lanes ? sm + lane * 33 : sm + lane;
            const int ps = rows_on_lanes ? 1 : 33;
            T* yp = y + sp * a.part;
#pragma unroll 4
            for (int i = 0; i < n; ++i, at += step) {
                float s = p[i * ps] + b;
                if (residual) s += ld1(residual + at);
                if (z) z[at] = from_float<T>(s);
                yp[at] = from_float<T>(act_run<kFast<T>>(s, a.act));
            }
        }
        __syncwarp();
    }
};

// grad_bias of one chunk of eight columns a warp: two threads' four columns, 16 threads' rows, joined in a fixed order.
// The sums are a few MB at most, and the warps that join them would wait for a product's first accumulator meanwhile: a
// launch of its own made the backward pass of 5000x2048x512 9 us longer. (Rows of `pitch`, a multiple of 8, are written
// to their ends.)
__device__ __forceinline__ void join_bias(const Sums& s, int chunk, int chunks, int lane) {
    for (; chunk * 8 < s.n; chunk += chunks) {
        const int n = chunk * 8 + lane % 2 * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 12
        for (int i = lane / 2; i < s.blocks; i += 16) {
            const float4 w = __ldg(reinterpret_cast<const float4*>(s.sums + (long long)i * s.pitch + n));
            v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
        }
#pragma unroll
        for (int d = 2; d < 32; d *= 2) {
            v.x += __shfl_xor_sync(~0u, v.x, d);
            v.y += __shfl_xor_sync(~0u, v.y, d);
            v.z += __shfl_xor_sync(~0u, v.z, d);
            v.w += __shfl_xor_sync(~0u, v.w, d);
        }
        // gb has no alignment of its own to rely on
        if (lane < 8) {
            const int k = lane / 2;
            const float one = k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
            if (n + k < s.n) s.gb[n + k] = one;
        }
    }
}

// T: element type of D. PB: 0, or BN where the accumulator is added up in registers.
template <typename T, int PB, int CG>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_tc_kernel(const __grid_constant__ CUtensorMap tma, const __grid_constant__ CUtensorMap tmb,
                   const __grid_constant__ CUtensorMap tmy, const __grid_constant__ CUtensorMap tmz,
                   const __grid_constant__ CUtensorMap tmr, const GemmArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = CG == 2 ? (int)ptx::cluster_ctarank() : 0;
    const int group = blockIdx.x / CG, groups = gridDim.x / CG;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + a.bar_off);
    const uint32_t full = ptx::smem_u32(bars), empty = full + MAX_STAGES * 8;
    const uint32_t accfull = empty + MAX_STAGES * 8, accempty = accfull + 16, done = accempty + 16;
    const uint32_t resbar = done + 8;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * MAX_STAGES + 5 + EPI_WARPS * MAX_SLOTS);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    const uint32_t base = ptx::smem_u32(smem);

    asm volatile("griddepcontrol.launch_dependents;");
    if (tid == 0) {
        for (int i = 0; i < MAX_STAGES; ++i) {
            ptx::mbar_init(full + i * 8, 2);  // both producers
            ptx::mbar_init(empty + i * 8, 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(accfull + i * 8, 1);
            ptx::mbar_init(accempty + i * 8, EPI_WARPS * CG);
        }
        ptx::mbar_init(done, 1);
        for (int i = 0; i < EPI_WARPS * MAX_SLOTS; ++i) ptx::mbar_init(resbar + i * 8, 1);
        *s_abort = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tma);
        ptx::prefetch_tmap(&tmb);
    }
    if (warp == 1) ptx::tmem_alloc_cg<CG>(ptx::smem_u32(s_tmem), TMEM_COLS);
    ptx::tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) ptx::cluster_sync();  // the pair's barriers are ready
    ptx::tc_fence_after();
    const uint32_t tmem = *s_tmem;
    // a programmatic dependent of the stream's previous work: nothing global is touched before it is complete
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int units = a.mt * a.nt * a.splits;
    // (32-bit divisions, and none where there is nothing to divide: 20000x1024x256 took 17.2 us with 64-bit ones, 14.4 so)
    auto unit_of = [&](int u, int& im, int& in, int& k0, int& k1, int& sp) {
        int t = u;
        sp = 0;
        k0 = 0;
        k1 = a.kblocks;
        if (a.splits > 1) {
            t = (int)((unsigned)u / (unsigned)a.splits);
            sp = u - t * a.splits;
            k0 = sp * a.kper + min(sp, a.kmore);
            k1 = k0 + a.kper + (sp < a.kmore);
        }
        im = t;
        in = 0;
        if (a.nt > 1) {
            im = (int)((unsigned)t / (unsigned)a.nt);
            in = t - im * a.nt;
        }
    };

    if (warp == 0 || warp == B_WARP) {
        // ---- TMA producers, one for each operand: this CTA's rows of A, its share of B's rows. The whole warp walks
        // the loop and one elected lane issues. (One warp for both took 640 cycles a stage, whatever its size: the
        // issue of a load costs about 200, and a stage's MMAs take 2 bn.)
        const bool isb = warp == B_WARP;
        const Operand& o = isb ? a.b : a.a;
        const CUtensorMap* map = isb ? &tmb : &tma;
        const int rows = isb ? a.bn / CG : BM;
        const uint32_t term_bytes = (uint32_t)rows * 128, bytes = term_bytes * o.terms;
        const uint32_t first = base + (isb ? a.a.terms * A_BYTES : 0);
        int stage = 0, it = 0;
        uint32_t phase = 1;  // of the empty barrier: the first round of stages is free
        bool ok = true;
        for (int u = group; u < units && ok; u += groups) {
            int im, in, k0, k1, sp;
            unit_of(u, im, in, k0, k1, sp);
            const int r0 = isb ? in * a.bn + rank * rows : (im * CG + rank) * BM;
            // coordinates: K-major (64 kb, row, 0), MN-major in one box (0, 64 kb, row / 64) or a box for each 64 rows
            // (row, 64 kb, 0)
            const int x0 = o.kind == kMnRows ? r0 : 0, dx = o.kind == kKMajor ? BK : 0;
            const int y0 = o.kind == kKMajor ? r0 : 0, dy = BK - dx, z0 = o.kind == kMnBlocks ? r0 / 64 : 0;
            for (int kb = k0; kb < k1; ++kb, ++it) {
                ok = ptx::mbar_wait(empty + stage * 8, phase, s_abort, a.status, WAIT_LIMIT);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                if (ptx::elect_one()) {
                    const uint32_t bar = full + stage * 8, dst = first + stage * a.stage_bytes;
                    if (rank == 0) ptx::mbar_arrive_expect_tx(bar, bytes * CG);
                    const int x = x0 + kb * dx, y = y0 + kb * dy;
                    if (o.kind != kMnRows) {
                        ptx::tma_load_4d_cg<CG>(dst, map, bar, x, y, z0, 0);
                        if (o.terms > 1) ptx::tma_load_4d_cg<CG>(dst + term_bytes, map, bar, x, y, z0, 1);
                        if (o.terms > 2) ptx::tma_load_4d_cg<CG>(dst + 2 * term_bytes, map, bar, x, y, z0, 2);
                    } else {
                        for (int t = 0; t < o.terms; ++t)
                            for (int h = 0; h < rows / 64; ++h)
                                ptx::tma_load_4d_cg<CG>(dst + t * term_bytes + h * MN_BLOCK, map, bar, x + h * 64, y, 0,
                                                        t);
                    }
                }
                __syncwarp();
                if (++stage == a.stages) stage = 0, phase ^= 1;
            }
        }
        // copies still in flight land before the CTA may exit (bounded)
        if (rank == 0 && lane == 0) {
            volatile int none = 0;
            for (int k = std::max(0, it - a.stages); k < it; ++k)
                ptx::mbar_wait(full + (k % a.stages) * 8, (k / a.stages) & 1, &none, nullptr, WAIT_LIMIT);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            // ---- MMA issue, by one elected lane. The loop keeps nothing that needs a division or a 64-bit sum per step
            const bool a_mn = a.a.kind != kKMajor, b_mn = a.b.kind != kKMajor;
            const uint32_t idesc =
                ptx::idesc_bf16_f32(BM * CG, a.bn) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16);
            const OperandDesc da(base, a_mn), db(base + a.a.terms * A_BYTES, b_mn);
            const uint32_t aterm = A_BYTES / 16, bterm = (uint32_t)(a.bn / CG) * 128 / 16;
            const uint32_t stage_units = a.stage_bytes / 16;
            const bool one = a.a.terms * a.b.terms == 1, two = a.a.terms * a.b.terms == 2, both = a.b.terms > 1;
            const uint32_t a2 = a.a.terms == 2 ? aterm : 0, b2 = aterm == a2 ? 0 : bterm;  // of two: the second product's
            int stage = 0;
            uint32_t phase = 0, acc_phase = 1, off = 0;
            int buf = 0;
            bool ok = true;
            for (int u = group; u < units && ok; u += groups) {
                int im, in, k0, k1, sp;
                unit_of(u, im, in, k0, k1, sp);
                for (int c0 = k0; c0 < k1 && ok; c0 += a.chunk) {
                    ok = ptx::mbar_wait(accempty + buf * 8, acc_phase, s_abort, a.status, WAIT_LIMIT);
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t acc = tmem + buf * 256, low = acc + 128;
                    const int c1 = min(c0 + a.chunk, k1);
                    for (int kb = c0; kb < c1; ++kb) {
                        ok = ptx::mbar_wait(full + stage * 8, phase, s_abort, a.status, WAIT_LIMIT);
                        ok = __all_sync(~0u, ok);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        if (ptx::elect_one()) {
                            const uint32_t first = kb > c0;
                            if (one) {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    ptx::mma_bf16_cg<CG>(acc, da.at(off, k), db.at(off, k), idesc, k ? 1u : first);
                            } else if (two) {  // a bfloat16 result: one accumulator for both
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    ptx::mma_bf16_cg<CG>(acc, da.at(off, k), db.at(off, k), idesc, k ? 1u : first);
                                    ptx::mma_bf16_cg<CG>(acc, da.at(off + a2, k), db.at(off + b2, k), idesc, 1u);
                                }
                            } else {
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const uint32_t more = k ? 1u : first;
                                    const uint64_t a0 = da.at(off, k), b0 = db.at(off, k);
                                    ptx::mma_bf16_cg<CG>(acc, a0, b0, idesc, more);
                                    const uint64_t a1 = da.at(off + aterm, k);
                                    ptx::mma_bf16_cg<CG>(low, a1, b0, idesc, more);
                                    ptx::mma_bf16_cg<CG>(low, da.at(off + 2 * aterm, k), b0, idesc, 1u);
                                    if (both) {
                                        const uint64_t b1 = db.at(off + bterm, k);
                                        ptx::mma_bf16_cg<CG>(low, a0, db.at(off + 2 * bterm, k), idesc, 1u);
                                        ptx::mma_bf16_cg<CG>(low, a1, b1, idesc, 1u);
                                        ptx::mma_bf16_cg<CG>(low, a0, b1, idesc, 1u);
                                    }
                                }
                            }
                            ptx::mma_commit_cg<CG>(empty + stage * 8);
                            if (kb + 1 == c1) ptx::mma_commit_cg<CG>(accfull + buf * 8);
                        }
                        __syncwarp();
                        off += stage_units;
                        if (++stage == a.stages) stage = 0, off = 0, phase ^= 1;
                    }
                    buf ^= 1;
                    acc_phase ^= buf ^ 1;
                }
            }
            // every issued MMA has completed before TMEM and shared memory are released (bounded)
            volatile int none = 0;
            if (ptx::elect_one()) ptx::mma_commit_cg<CG>(done);
            __syncwarp();
            ptx::mbar_wait(done, 0, &none, a.status, WAIT_LIMIT);
        }
    } else {
        // ---- epilogue: quarter q of the lanes, part h of the columns (a part is a whole chunk at least)
        constexpr int COLS = Emit<T>::COLS;
        const int w = warp - 2, q = warp & 3, h = w >> 2;
        const int half = max(a.bn / 2, COLS), nch = h * half < a.bn ? half / COLS : 0;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + h * half;
        int buf = 0;
        uint32_t phase = 0;
        Emit<T> emit{a, &tmy, &tmz, &tmr, (T*)a.y, (T*)a.z, (const T*)a.bias, (const T*)a.residual};
        emit.slots = base + a.slot_off + w * (a.nslots * SLOT_BYTES);
        emit.resbar = resbar + w * (MAX_SLOTS * 8);
        emit.sm = reinterpret_cast<float*>(smem + a.slot_off + w * EXCHANGE_BYTES);
        emit.sbias = reinterpret_cast<float*>(smem + a.sm_off + w * BIAS_BYTES);
        emit.abort = s_abort;
        emit.lane = lane;
        auto place = [&](int u, int& row, int& col, int& k0, int& k1, int& sp) {
            int im, in;
            unit_of(u, im, in, k0, k1, sp);
            row = (im * CG + rank) * BM + q * 32;
            col = in * a.bn + h * half;
        };
        auto wait_acc = [&]() {
            const bool ok = ptx::mbar_wait(accfull + buf * 8, phase, s_abort, a.status, WAIT_LIMIT);
            const bool all = __all_sync(~0u, ok && emit.ok);
            ptx::tc_fence_after();
            return all;
        };
        auto free_acc = [&]() {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_cg<CG>(accempty + buf * 8);
            buf ^= 1;
            phase ^= buf ^ 1;
        };
        if (a.gb.gb) join_bias(a.gb, w * gridDim.x + blockIdx.x, EPI_WARPS * gridDim.x, lane);
        // the residual's cursor: the next chunk to fetch, nslots - 1 ahead of the one written
        const bool has_res = a.residual && a.tma_out;
        int fu = group, fc = 0;
        auto fetch_next = [&]() {
            while (fu < units) {
                int row, col, k0, k1, sp;
                place(fu, row, col, k0, k1, sp);
                col += fc * COLS;
                const bool there = nch > 0 && emit.active(row, col);
                if (++fc >= nch) fc = 0, fu += groups;
                if (there) {
                    emit.fetch(row, col);
                    return;
                }
            }
        };
        if (has_res)
            for (int i = 0; i < a.nslots - 1; ++i) fetch_next();
        // the bias of a tile is loaded while the tile before is written
        const bool has_bias = a.bias && a.tma_out;
        float bnext[4] = {};
        auto load_bias = [&](int u) {
            int row, col, k0, k1, sp;
            place(u, row, col, k0, k1, sp);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                bnext[i] = i * 32 < half && col + i * 32 + lane < a.cols ? ld1((const T*)a.bias + col + i * 32 + lane) : 0.f;
        };
        if (has_bias && group < units) load_bias(group);
        for (int u = group; u < units; u += groups) {
            int row, col, k0, k1, sp;
            place(u, row, col, k0, k1, sp);
            emit.row0 = row;
            emit.sp = sp;
            if (has_bias) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) emit.sbias[i * 32 + lane] = bnext[i];
                __syncwarp();
                if (u + groups < units) load_bias(u + groups);
            }
            auto write = [&](float(&v)[COLS], int c) {
                const int before = emit.out;
                emit.chunk(v, col + c * COLS, c * COLS, std::is_same<T, bf16>::value || (PB != 0 && PB != 256));
                if (has_res && emit.out != before) {
                    emit.freed();
                    fetch_next();
                }
            };
            if constexpr (PB == 0) {
                if (!wait_acc()) break;
                const uint32_t acc = lanes + buf * 256;
                if (nch == 0) free_acc();
                for (int c = 0; c < nch; ++c) {
                    float v[COLS];
                    uint32_t r[COLS / 32][32];
#pragma unroll
                    for (int i = 0; i < COLS / 32; ++i) ptx::tmem_ld32_issue(acc + c * COLS + i * 32, r[i]);
#pragma unroll
                    for (int i = 0; i < COLS / 32; ++i) ptx::tmem_wait_ld(r[i]);
                    if (c + 1 == nch) free_acc();
#pragma unroll
                    for (int i = 0; i < COLS; ++i) v[i] = __uint_as_float(r[i / 32][i % 32]);
                    write(v, c);
                }
            } else {
                constexpr int HALF = PB / 2 > COLS ? PB / 2 : COLS;
                float acc[HALF] = {};
                bool ok = true;
                for (int c0 = k0; c0 < k1; c0 += a.chunk) {
                    ok = wait_acc();
                    if (!ok) break;
                    const uint32_t from = lanes + buf * 256;
#pragma unroll
                    for (int j = 0; j < HALF; j += 32) {
                        if (PB == 64 && HALF == PB && nch == 0) break;
                        float v[32];
                        ptx::tmem_ld32(from + j, v);
                        if (std::is_same<T, float>::value && PB <= 128 && a.a.terms > 2) {
                            float l[32];
                            ptx::tmem_ld32(from + 128 + j, l);
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float sum = v[i] + l[i];
                                v[i] = fabsf(v[i]) <= 3.4028234663852886e38f ? sum : v[i];
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) acc[j + i] += v[i];
                    }
                    free_acc();
                }
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < HALF; j += COLS)
                    if (!(PB == 64 && HALF == PB && nch == 0)) write(*reinterpret_cast<float(*)[COLS]>(&acc[j]), j / COLS);
            }
        }
        // residual chunks asked for have landed, and stores have read their slots, before the CTA leaves (bounded)
        if (has_res)
            for (int i = emit.out; i < emit.in; ++i) {
                volatile int none = 0;
                ptx::mbar_wait(emit.resbar + (i % a.nslots) * 8, (i / a.nslots) & 1, &none, a.status, WAIT_LIMIT);
            }
        if (lane == 0) ptx::bulk_wait_group_read<0>();
        __syncwarp();
    }

    ptx::tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) ptx::cluster_sync();  // neither CTA leaves while the other may signal or read it
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc_cg<CG>(tmem, TMEM_COLS);
    }
}

// -------------------------------------------------- after the products --

// What remains after a split reduction: its parts are joined.
template <typename T>
struct FinishArgs {
    // D[m, n] = sum of the parts (in order), then the epilogue; four columns a thread
    const float* part;
    long long stride;  // elements between two parts
    int splits, M, N, pitch, part_blocks;
    const T *bias, *residual;
    T *y, *z;
    int act;
};

constexpr int FINISH_THREADS = 256;

template <typename T>
__global__ void __launch_bounds__(FINISH_THREADS) finish_kernel(const FinishArgs<T> a) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n4 = (a.N + 3) / 4;
    const long long total = (long long)a.M * n4;
    for (long long i = blockIdx.x * (long long)FINISH_THREADS + threadIdx.x; i < total;
         i += (long long)a.part_blocks * FINISH_THREADS) {
        const long long m = i / n4;
        const int n = (int)(i - m * n4) * 4;
        const float* p = a.part + m * a.pitch + n;
        float v[4] = {};
#pragma unroll 10
        for (int s = 0; s < a.splits; ++s) {
            const float4 q = *reinterpret_cast<const float4*>(p + s * a.stride);
            v[0] += q.x, v[1] += q.y, v[2] += q.z, v[3] += q.w;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (n + c < a.N) {
                const long long at = m * a.N + n + c;
                float s = v[c];
                if (a.bias) s += ld1(a.bias + n + c);
                if (a.residual) s += ld1(a.residual + at);
                if (a.z) a.z[at] = from_float<T>(s);
                a.y[at] = from_float<T>(act_run<kFast<T>>(s, a.act));
            }
    }
}

// grad_bias by itself, where no product is asked for.
__global__ void __launch_bounds__(32) bias_kernel(const Sums s) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    join_bias(s, blockIdx.x, gridDim.x, threadIdx.x);
}

// ----------------------------------------------------- operand preparation --

// The three bfloat16 terms of v. The first is kept finite for a finite v, the others are zero
// for an infinite or NaN v.
__device__ __forceinline__ void split3(float v, bf16 (&t)[3]) {
    const float top = 3.3895313892515355e38f;  // the largest bfloat16
    const bool fin = fabsf(v) <= 3.4028234663852886e38f;
    t[0] = __float2bfloat16_rn(fin ? fminf(fmaxf(v, -top), top) : v);
    const float r1 = fin ? v - __bfloat162float(t[0]) : 0.f;
    t[1] = __float2bfloat16_rn(r1);
    t[2] = __float2bfloat16_rn(r1 - __bfloat162float(t[1]));
}

// Eight values from p, `n` of them there (the others 0); VEC: all there, 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ void load8(float (&v)[8], const float* p, int n) {
    if constexpr (VEC) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = q < n ? ld1(p + q) : 0.f;
    }
}
template <bool VEC>
__device__ __forceinline__ void load8(float (&v)[8], const bf16* p, int n) {
    if constexpr (VEC) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = __uint_as_float(w[q] << 16);
            v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = q < n ? ld1(p + q) : 0.f;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
    return *reinterpret_cast<uint4*>(h);
}

template <bool VEC>
__device__ __forceinline__ void store8(float* p, const float (&v)[8], int n) {
    if constexpr (VEC) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < n) p[q] = v[q];
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(bf16* p, const float (&v)[8], int n) {
    if constexpr (VEC) {
        *reinterpret_cast<uint4*>(p) = pack8(v);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < n) p[q] = __float2bfloat16_rn(v[q]);
    }
}

// The TERMS bfloat16 terms of eight values to out, out + plane, ...
template <int TERMS>
__device__ __forceinline__ void store_terms(bf16* out, long long plane, const float (&v)[8]) {
    if constexpr (TERMS == 1) {
        *reinterpret_cast<uint4*>(out) = pack8(v);
    } else {
        float most = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) most = fmaxf(most, fabsf(v[q]));
        if (most < 3.38e38f) {  // none infinite, nor rounded to infinity (a NaN may stay one in every term)
            float r[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) r[q] = v[q];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const uint4 t = pack8(r);
                *reinterpret_cast<uint4*>(out + k * plane) = t;
                const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    r[2 * q] -= __uint_as_float(w[q] << 16);
                    r[2 * q + 1] -= __uint_as_float(w[q] & 0xFFFF0000u);
                }
            }
            return;
        }
        bf16 t[3][8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            bf16 s[3];
            split3(v[q], s);
#pragma unroll
            for (int k = 0; k < 3; ++k) t[k][q] = s[k];
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4*>(out + k * plane) = *reinterpret_cast<uint4*>(t[k]);
    }
}

// out[term][r][c] (bfloat16, rows of `pitch`) = the terms of in[r][c]; eight columns a thread.
// vec: rows of `in` are whole vectors, 16-byte aligned.
template <typename T>
struct PackJob {
    const T* in;
    int rows, cols, pitch, vec, blocks;
    bf16* out;
};
// dz = grad_y act'(saved): its bfloat16 terms (out, as PackJob; may be null), grad_residual (may be null), and the
// column sums of a block's rows (sums[row block][pitch]; may be null). A thread keeps eight columns and walks the
// block's rows. vec as for PackJob, for gy, saved and gr.
template <typename T>
struct DzJob {
    const T *gy, *saved;
    int M, N, pitch, rows, cblocks, vec, blocks;
    bf16* out;
    T* gr;
    float* sums;
};

template <typename T, bool VEC>
__device__ __forceinline__ void run_pack(const PackJob<T>& j, int block) {
    constexpr int TERMS = std::is_same<T, bf16>::value ? 1 : 3;
    const int c8 = j.pitch / 8;
    const long long plane = (long long)j.rows * j.pitch;
    for (long long i = block * 256LL + threadIdx.x; i < (long long)j.rows * c8; i += j.blocks * 256LL) {
        const long long r = i / c8;
        const int c = (int)(i - r * c8) * 8;
        float v[8];
        load8<VEC>(v, j.in + r * j.cols + c, j.cols - c);
        store_terms<TERMS>(j.out + r * j.pitch + c, plane, v);
    }
}

constexpr int SUM_PITCH = 260;  // of a block's partial column sums: no bank conflicts, written or read

template <typename T, int ACT, int TERMS, bool VEC>
__device__ __forceinline__ void run_dz(const DzJob<T>& j, int block, float* sm) {
    const int c8 = j.pitch / 8;
    const int tx = min(c8, 256), ty = 256 / tx;
    const int cx = threadIdx.x % tx, ry = threadIdx.x / tx;
    const int rb = block / j.cblocks;
    const int c = ((block % j.cblocks) * tx + cx) * 8;
    const long long plane = (long long)j.M * j.pitch;
    const int m0 = rb * j.rows, m1 = min(m0 + j.rows, j.M);
    float sum[8] = {};
    if (c < j.pitch && ry < ty) {
#pragma unroll 4
        for (long long m = m0 + ry; m < m1; m += ty) {
            const long long at = m * j.N + c;
            float v[8];
            load8<VEC>(v, j.gy + at, j.N - c);
            if constexpr (ACT != kActNone) {
                float s[8];
                load8<VEC>(s, j.saved + at, j.N - c);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = act_grad<ACT, kFast<T>>(v[q], s[q]);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) sum[q] += v[q];
            if (j.gr) store8<VEC>(j.gr + at, v, j.N - c);
            if (j.out) store_terms<TERMS>(j.out + m * j.pitch + c, plane, v);
        }
    }
    if (!j.sums) return;
#pragma unroll
    for (int q = 0; q < 8; ++q) sm[q * SUM_PITCH + threadIdx.x] = sum[q];
    __syncthreads();
    const int c0 = (block % j.cblocks) * tx * 8;
    for (int i = threadIdx.x; i < tx * 8; i += 256) {  // a column each
        float v = 0.f;
        for (int r = 0; r < ty; ++r) v += sm[(i % 8) * SUM_PITCH + r * tx + i / 8];
        if (c0 + i < j.pitch) j.sums[(long long)rb * j.pitch + c0 + i] = v;
    }
}

// All of a call's operand preparation in one launch.
template <typename T, int ACT, int TERMS>
__global__ void __launch_bounds__(256) prep_kernel(const DzJob<T> dz, const PackJob<T> a, const PackJob<T> b) {
    __shared__ float sm[SUM_PITCH * 8];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int block = blockIdx.x;
    if (block < dz.blocks) {
        if (dz.vec) run_dz<T, ACT, TERMS, true>(dz, block, sm);
        else run_dz<T, ACT, TERMS, false>(dz, block, sm);
        return;
    }
    block -= dz.blocks;
    const PackJob<T>& j = block < a.blocks ? a : b;
    if (block >= a.blocks) block -= a.blocks;
    if (j.vec) run_pack<T, true>(j, block);
    else run_pack<T, false>(j, block);
}

// ------------------------------------------------------------------- host --

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// A bfloat16 matrix in memory, [terms][rows][pitch]: 16-byte aligned, pitch a multiple of 8.
struct Matrix {
    const void* p;
    int rows, cols, pitch, terms;
};

// Its tensor map for `rows` operand rows a stage. K-major: boxes of 64 reduction elements and `rows` rows. MN-major:
// 64 reduction rows and 64 operand rows (128 bytes) a block; where the blocks tile the matrix exactly, they are a
// dimension of their own and one box holds all of a stage's.
bool encode(CUtensorMap* m, const Matrix& x, bool mn, int rows, int* kind) {
    const auto fn = encode_fn();
    if (!fn) return false;
    const bool blocks = mn && x.cols % 64 == 0;
    *kind = !mn ? kKMajor : blocks ? kMnBlocks : kMnRows;
    cuuint64_t dims[4] = {(cuuint64_t)(blocks ? 64 : x.cols), (cuuint64_t)x.rows, (cuuint64_t)(blocks ? x.cols / 64 : 1),
                          (cuuint64_t)x.terms};
    const cuuint64_t plane = (cuuint64_t)x.pitch * 2 * x.rows;
    cuuint64_t strides[3] = {(cuuint64_t)x.pitch * 2, blocks ? 128 : plane, plane};
    cuuint32_t b[4] = {64, (cuuint32_t)(mn ? BK : rows), (cuuint32_t)(blocks ? rows / 64 : 1), 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(x.p), dims, strides, b, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The map of a result's chunks (128 bytes of 32 rows): [parts][rows][pitch] of T.
template <typename T>
bool encode_out(CUtensorMap* m, const void* p, int rows, int cols, int pitch, int parts) {
    const auto fn = encode_fn();
    if (!fn) return false;
    constexpr bool f32 = std::is_same<T, float>::value;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)parts};
    cuuint64_t strides[2] = {(cuuint64_t)pitch * sizeof(T), (cuuint64_t)pitch * sizeof(T) * rows};
    cuuint32_t b[3] = {128 / sizeof(T), 32, 1}, es[3] = {1, 1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims,
              strides, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename... P, typename... Q>
cudaError_t launch(void (*f)(P...), int grid, int threads, uint32_t smem, int cluster, cudaStream_t st, Q... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, f, P(args)...);
}

// How one product runs.
struct GemmPlan {
    bool swap;  // D's columns on the lanes
    int cg, bn, splits, chunk;
};

// The cheapest of the tilings by a model of one CTA's cycles: per stage the larger of the MMAs (bn / 2
// cycles each, but 75 to issue one, and 150 to wait and commit) and the operands' bytes from L2 (56 a cycle), per tile the
// result's bytes (24 a cycle, an SM's share of HBM) with the activation's cost and 700 cycles of its own, and the
// parts' way through L2 and a second launch where the reduction is split (grad_weight of 20000x256x1024: 18 parts of
// 256 x 256 tiles 24.8 us, nine of 256 x 128 22.8 us).
GemmPlan plan_gemm(long long rows, long long cols, int red, int ta, int tb, bool f32_out, int out_bytes, int act) {
    const int kblocks = (red + BK - 1) / BK;
    const int sms = num_sms();
    const int prods = tb == 1 ? ta : 6;
    const double element = out_bytes / 24.0 + (act == kActSilu || act == kActGelu ? 0.2 : 0.0);
    GemmPlan best = {};
    double best_t = 1e300;
    for (int swap = 0; swap < 2; ++swap) {
        const long long r = swap ? cols : rows, c = swap ? rows : cols;
        const int sa = swap ? tb : ta, sb = swap ? ta : tb;
        if (sa < sb && sb > 2) continue;  // the kernel takes the operand in three terms as A
        for (int cg = 1; cg <= 2; ++cg)
            for (int bn = 64; bn <= (prods > 2 ? 128 : 256); bn *= 2) {
                if (cg == 2 && bn < 128) continue;
                if (bn > 64 && bn / 2 >= c) continue;
                if (prods == 6 && cg == 1 && bn == 128) continue;  // shared memory holds one stage only
                const long long mt = (r + BM * cg - 1) / (BM * cg), nt = (c + bn - 1) / bn;
                const int slots = sms / cg;
                const double stage = std::max(4.0 * prods * std::max(bn / 2.0, 75.0) + 150.0,
                                              (sa * (double)A_BYTES + sb * bn / cg * 128.0) / 56.0);
                const double epi = BM * (double)bn * (swap ? 2.0 : 1.0) * element, part = BM * bn * (swap ? 3.0 : 1.0) * 4 / 20.0;
                // no split, or as many parts as fill the GPU once, or half of them
                const int fill = (int)std::min<long long>(kblocks, std::max<long long>(1, slots / (mt * nt)));
                int last = 0;
                for (const int splits : {1, fill / 2, fill}) {
                    if (splits <= last) continue;
                    last = splits;
                    const long long waves = (mt * nt * splits + slots - 1) / slots;
                    const int kb = (kblocks + splits - 1) / splits;
                    double t = waves * (std::max(kb * stage, splits > 1 ? part : epi) + 700.0) +
                               (splits > 1 ? part : epi) + 2000.0;
                    if (splits > 1) t += 4000.0 + (double)rows * cols * (4.0 * splits + out_bytes) / (sms * 12.0);
                    // (on a tie pairs, for the L2's sake: grad_x of 5000x2048x512 silu 45 us, with single CTAs 53)
                    if (t < best_t || (t == best_t && cg > best.cg)) {
                        best_t = t;
                        best = {swap != 0, cg, bn, splits, 0};
                    }
                }
            }
    }
    // float32 results: the accumulator is taken out every 256 (terms: 128) elements; bfloat16 results of reductions over
    // LONG stages in equal pieces of up to so many
    const int part = (kblocks + best.splits - 1) / best.splits, pieces = (part + LONG - 1) / LONG;
    best.chunk = f32_out ? (prods > 1 ? 2 : 4) : pieces > 1 ? (part + pieces - 1) / pieces : 1 << 28;
    return best;
}

template <typename T, int PB, int CG>
cudaError_t launch_gemm(const CUtensorMap (&m)[5], const GemmArgs& a, int grid, uint32_t smem, cudaStream_t st) {
    static DeviceFlags attr;
    cudaError_t e = max_dynamic_smem_once((const void*)gemm_tc_kernel<T, PB, CG>, SMEM_MAX, attr);
    if (e != cudaSuccess) return e;
    return launch(gemm_tc_kernel<T, PB, CG>, grid, THREADS, smem, CG, st, m[0], m[1], m[2], m[3], m[4], a);
}

template <typename T>
struct Out {  // the result's epilogue
    const T *bias, *residual;
    T *y, *z;
    int act;
};

size_t part_bytes(const GemmPlan& p, long long rows, long long cols) {
    return p.splits > 1 ? (size_t)p.splits * rows * ((cols + 7) / 8 * 8) * 4 : 0;
}

template <typename T>
cudaError_t finish(const FinishArgs<T>& f, cudaStream_t st, int* launches) {
    ++*launches;
    return launch(finish_kernel<T>, f.part_blocks, FINISH_THREADS, 0, 1, st, f);
}

// D [rows, cols] (rows of `cols`) = A B^T through the epilogue, and (sums) grad_bias beside it. A: K-major [rows, red], or (a_mn) [red, rows]; B alike
// with cols. `parts`: room for the split reduction's results.
template <typename T>
cudaError_t run_gemm(const GemmPlan& p, const Matrix& A, bool a_mn, const Matrix& B, bool b_mn, int rows, int cols,
                     int red, const Out<T>& out, float* parts, bool f32_out, const Sums& sums, unsigned* status,
                     cudaStream_t st, int* launches) {
    const Matrix &L = p.swap ? B : A, &R = p.swap ? A : B;
    const bool l_mn = p.swap ? b_mn : a_mn, r_mn = p.swap ? a_mn : b_mn;
    GemmArgs a = {};
    a.rows = p.swap ? cols : rows;
    a.cols = p.swap ? rows : cols;
    a.kblocks = (red + BK - 1) / BK;
    a.splits = p.splits;
    a.kper = a.kblocks / p.splits;
    a.kmore = a.kblocks % p.splits;
    a.chunk = p.chunk;
    a.mt = (a.rows + BM * p.cg - 1) / (BM * p.cg);
    a.nt = (a.cols + p.bn - 1) / p.bn;
    a.bn = p.bn;
    a.a.terms = L.terms;
    a.b.terms = R.terms;
    a.stage_bytes = L.terms * A_BYTES + R.terms * (uint32_t)(p.bn / p.cg) * 128;
    a.status = status;
    a.gb = sums;
    a.one_column = cols == 1;
    const bool split = p.splits > 1;
    const int pitch = split ? (cols + 7) / 8 * 8 : cols;
    a.rs = p.swap ? 1 : pitch;
    a.cs = p.swap ? pitch : 1;
    a.part = (long long)rows * pitch;
    if (split) {
        a.y = parts;
        a.tma_out = !p.swap;
    } else {
        a.bias = out.bias;
        a.residual = out.residual;
        a.y = out.y;
        a.z = out.z;
        a.act = out.act;
        const uintptr_t all = (uintptr_t)out.y | (uintptr_t)out.z | (uintptr_t)out.residual | (uintptr_t)(pitch * sizeof(T));
        a.tma_out = !p.swap && all % 16 == 0;
    }
    // Two slots a warp, so that one is written while the other is stored; a third lets the residual run two chunks
    // ahead. Long reductions, whose epilogue is rare, leave the room to the operands' stages.
    if (a.residual)
        a.nslots = a.kblocks <= 8 && L.terms == 1 ? 3 : 2;
    else
        a.nslots = a.kblocks <= 16 && L.terms == 1 ? 2 : 1;
    const uint32_t epi = EPI_WARPS * (a.tma_out ? a.nslots * SLOT_BYTES : EXCHANGE_BYTES);
    const uint32_t extra = epi + BAR_BYTES + EPI_WARPS * BIAS_BYTES;
    a.stages = (int)std::min<uint32_t>(MAX_STAGES, (SMEM_MAX - 1024 - extra) / a.stage_bytes);
    a.slot_off = a.stages * a.stage_bytes;
    a.bar_off = a.slot_off + epi;
    a.sm_off = a.bar_off + BAR_BYTES;
    if (a.stages < 1) return cudaErrorInvalidConfiguration;
    CUtensorMap m[5] = {};
    if (!encode(&m[0], L, l_mn, BM, &a.a.kind) || !encode(&m[1], R, r_mn, p.bn / p.cg, &a.b.kind))
        return cudaErrorInvalidValue;
    if (a.tma_out) {
        bool good = split ? encode_out<float>(&m[2], parts, rows, cols, pitch, p.splits)
                          : encode_out<T>(&m[2], out.y, rows, cols, pitch, 1);
        if (a.z) good = good && encode_out<T>(&m[3], out.z, rows, cols, pitch, 1);
        if (a.residual) good = good && encode_out<T>(&m[4], out.residual, rows, cols, pitch, 1);
        if (!good) return cudaErrorInvalidValue;
    }
    const long long units = (long long)a.mt * a.nt * a.splits;
    const int grid = (int)std::min<long long>(units, num_sms() / p.cg) * p.cg;
    const uint32_t smem = a.slot_off + extra + 1024;
    cudaError_t e;
    auto go = [&](auto t, auto pb) {
        using D = decltype(t);
        constexpr int PB = decltype(pb)::value;
        return p.cg == 2 ? launch_gemm<D, PB, 2>(m, a, grid, smem, st)
                         : launch_gemm<D, PB, 1>(m, a, grid, smem, st);
    };
    const bool taken = !f32_out && p.chunk < a.kblocks;  // out of the accumulator, on the way
    if (taken && !split) {
        e = p.bn == 64    ? go(T{}, std::integral_constant<int, 64>{})
            : p.bn == 128 ? go(T{}, std::integral_constant<int, 128>{})
                          : go(T{}, std::integral_constant<int, 256>{});
    } else if (f32_out || taken) {
        e = p.bn == 64    ? go(float{}, std::integral_constant<int, 64>{})
            : p.bn == 128 ? go(float{}, std::integral_constant<int, 128>{})
                          : go(float{}, std::integral_constant<int, 256>{});
    } else if (split) {
        e = go(float{}, std::integral_constant<int, 0>{});
    } else {
        e = go(T{}, std::integral_constant<int, 0>{});
    }
    if (e != cudaSuccess) return e;
    ++*launches;
    if (split) {
        FinishArgs<T> f = {};
        f.part = parts;
        f.stride = a.part;
        f.splits = p.splits;
        f.M = rows;
        f.N = cols;
        f.pitch = pitch;
        f.part_blocks = (int)std::min<long long>(((long long)rows * ((cols + 3) / 4) + FINISH_THREADS - 1) / FINISH_THREADS,
                                                 num_sms() * 8);
        f.bias = out.bias;
        f.residual = out.residual;
        f.y = out.y;
        f.z = out.z;
        f.act = out.act;
        return finish(f, st, launches);
    }
    return cudaSuccess;
}

int up8(int v) { return (v + 7) / 8 * 8; }
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// What a call lays out in its workspace.
struct FwdPlan {
    bool pack_x, pack_w;
    GemmPlan g;
    size_t x, w, parts, total;
};
FwdPlan plan_forward(const LinearShape& s, int bf) {
    FwdPlan p = {};
    const int terms = bf ? 1 : 3;
    bool xw, gy;
    linear_tc_in_place(s, bf, &xw, &gy);
    p.pack_x = p.pack_w = !xw;
    p.g = plan_gemm(s.M, s.N, s.K, terms, terms, !bf, bf ? 2 : 4, s.act);
    size_t o = 0;
    p.x = o;
    if (p.pack_x) o = up256(o + (size_t)terms * s.M * up8(s.K) * 2);
    p.w = o;
    if (p.pack_w) o = up256(o + (size_t)terms * s.N * up8(s.K) * 2);
    p.parts = o;
    p.total = o + part_bytes(p.g, s.M, s.N);
    return p;
}

struct BwdPlan {
    bool pack_x, pack_w, pass_dz;  // pass_dz: dz goes through the workspace
    int dz_terms, tx, ty, cblocks, rblocks, rows;
    GemmPlan gx, gw;
    size_t x, w, dz, sums, parts, total;
};
// How many bfloat16 terms of dz grad_weight, a float32 result, takes. dz is exact in one where it is grad_y or 0.
// (Two for silu and gelu leave out 2^-18 of it: 5000x2048x512 took 67.6 us without grad_bias, with three 73.5, but
// grad_weight was 10 times as far from the exact one.)
constexpr int dz_terms(int bf, bool smooth) { return bf && !smooth ? 1 : 3; }

// And how many grad_x takes: the two first of three for a bfloat16 result, whose rounding hides the third (2^-18 of dz).
// (With dz rounded to one, the backward of 5000x2048x512 gelu takes 78.6 us instead of 87.9, but grad_x is 1.4 to 1.5 times
// as far from the exact one.)
constexpr int gx_terms(int bf, bool smooth) { return bf ? (smooth ? 2 : 1) : 3; }

BwdPlan plan_backward(const LinearShape& s, int bf) {
    BwdPlan p = {};
    const int terms = bf ? 1 : 3;
    const bool smooth = s.act == kActSilu || s.act == kActGelu;
    bool xw, gy;
    linear_tc_in_place(s, bf, &xw, &gy);
    p.pack_x = p.pack_w = !xw;
    p.pass_dz = !gy;
    p.dz_terms = dz_terms(bf, smooth);
    p.gx = plan_gemm(s.M, s.K, s.N, gx_terms(bf, smooth), terms, !bf, bf ? 2 : 4, kActNone);
    p.gw = plan_gemm(s.N, s.K, s.M, p.dz_terms, terms, true, 4, kActNone);
    const int c8 = up8(s.N) / 8;
    p.tx = std::min(c8, 256);
    p.ty = 256 / p.tx;
    p.cblocks = (c8 + p.tx - 1) / p.tx;
    long long want = std::max(1, num_sms() * 4 / p.cblocks);
    want = std::min<long long>(want, (s.M + 4LL * p.ty - 1) / (4LL * p.ty));
    p.rows = (int)((s.M + want - 1) / want);
    p.rblocks = (s.M + p.rows - 1) / p.rows;
    size_t o = 0;
    p.x = o;
    if (p.pack_x) o = up256(o + (size_t)terms * s.M * up8(s.K) * 2);
    p.w = o;
    if (p.pack_w) o = up256(o + (size_t)terms * s.N * up8(s.K) * 2);
    p.dz = o;
    if (p.pass_dz) o = up256(o + (size_t)p.dz_terms * s.M * up8(s.N) * 2);
    p.sums = o;
    o = up256(o + (size_t)p.rblocks * up8(s.N) * 4);
    p.parts = o;
    p.total = o + std::max(part_bytes(p.gx, s.M, s.K), part_bytes(p.gw, s.N, s.K));
    return p;
}

template <typename T>
PackJob<T> pack_job(const T* in, int rows, int cols, void* out) {
    const int pitch = up8(cols);
    const long long n = ((long long)rows * (pitch / 8) + 255) / 256;
    return {in, rows, cols, pitch, cols % 8 == 0 && ((uintptr_t)in & 15) == 0,
            (int)std::min<long long>(n, num_sms() * 16), (bf16*)out};
}

template <typename T>
cudaError_t prepare(int act, const DzJob<T>& dz, const PackJob<T>& a, const PackJob<T>& b, cudaStream_t st,
                    int* launches) {
    const int blocks = dz.blocks + a.blocks + b.blocks;
    if (!blocks) return cudaSuccess;
    ++*launches;
    return with_act(dz.blocks ? act : kActNone, [&](auto A) {
        constexpr int ACT = decltype(A)::value;
        constexpr int TERMS = dz_terms(std::is_same<T, bf16>::value, ACT == kActSilu || ACT == kActGelu);
        return launch(prep_kernel<T, ACT, TERMS>, blocks, 256, 0, 1, st, dz, a, b);
    });
}

template <typename T>
cudaError_t forward_t(const LinearShape& s, const T* x, const T* w, const T* bias, const T* residual, T* y, T* z,
                      uint8_t* ws, unsigned* status, cudaStream_t st, int* launches) {
    constexpr int bf = std::is_same<T, bf16>::value;
    const FwdPlan p = plan_forward(s, bf);
    const int terms = bf ? 1 : 3;
    Matrix X{x, s.M, s.K, s.K, 1}, W{w, s.N, s.K, s.K, 1};
    PackJob<T> jx = {}, jw = {};
    if (p.pack_x) {
        jx = pack_job(x, s.M, s.K, ws + p.x);
        X = {ws + p.x, s.M, s.K, up8(s.K), terms};
    }
    if (p.pack_w) {
        jw = pack_job(w, s.N, s.K, ws + p.w);
        W = {ws + p.w, s.N, s.K, up8(s.K), terms};
    }
    const cudaError_t e = prepare<T>(kActNone, DzJob<T>{}, jx, jw, st, launches);
    if (e != cudaSuccess) return e;
    return run_gemm<T>(p.g, X, false, W, false, s.M, s.N, s.K, Out<T>{bias, residual, y, z, s.act},
                       (float*)(ws + p.parts), !bf, Sums{}, status, st, launches);
}

template <typename T>
cudaError_t backward_t(const LinearShape& s, const T* x, const T* w, const T* saved, const T* gy, T* gx, float* gw,
                       float* gb, T* gr, uint8_t* ws, unsigned* status, cudaStream_t st, int* launches) {
    constexpr int bf = std::is_same<T, bf16>::value;
    const BwdPlan p = plan_backward(s, bf);
    const int terms = bf ? 1 : 3;
    Matrix X{x, s.M, s.K, s.K, 1}, W{w, s.N, s.K, s.K, 1}, DZ{gy, s.M, s.N, s.N, 1};
    bf16* dz = p.pass_dz && (gx || gw) ? (bf16*)(ws + p.dz) : nullptr;
    DzJob<T> jd = {};
    PackJob<T> jx = {}, jw = {};
    if (dz || gb || gr) {
        jd = {gy,  saved, s.M, s.N, up8(s.N), p.rows, p.cblocks,
              s.N % 8 == 0 && (((uintptr_t)gy | (uintptr_t)saved | (uintptr_t)gr) & 15) == 0,
              p.rblocks * p.cblocks, dz, gr, gb ? (float*)(ws + p.sums) : nullptr};
        if (dz) DZ = {dz, s.M, s.N, up8(s.N), p.dz_terms};
    }
    if (gx && p.pack_w) {
        jw = pack_job(w, s.N, s.K, ws + p.w);
        W = {ws + p.w, s.N, s.K, up8(s.K), terms};
    }
    if (gw && p.pack_x) {
        jx = pack_job(x, s.M, s.K, ws + p.x);
        X = {ws + p.x, s.M, s.K, up8(s.K), terms};
    }
    cudaError_t e = prepare<T>(s.act, jd, jx, jw, st, launches);
    if (e != cudaSuccess) return e;
    const Sums sums{(const float*)(ws + p.sums), p.rblocks, up8(s.N), s.N, gb};
    if (gx) {
        Matrix first = DZ;
        first.terms = gx_terms(bf, s.act == kActSilu || s.act == kActGelu);
        e = run_gemm<T>(p.gx, first, false, W, true, s.M, s.K, s.N, Out<T>{nullptr, nullptr, gx, nullptr, kActNone},
                        (float*)(ws + p.parts), !bf, gw ? Sums{} : sums, status, st, launches);
        if (e != cudaSuccess) return e;
    }
    if (gw)
        return run_gemm<float>(p.gw, DZ, true, X, true, s.N, s.K, s.M,
                               Out<float>{nullptr, nullptr, gw, nullptr, kActNone}, (float*)(ws + p.parts), true, sums,
                               status, st, launches);
    if (gb && !gx) {
        ++*launches;
        return launch(bias_kernel, std::min((s.N + 7) / 8, 1 << 16), 32, 0, 1, st, sums);
    }
    return cudaSuccess;
}

}  // namespace

void linear_tc_in_place(const LinearShape& s, int bf, bool* in_xw, bool* in_gy) {
    *in_xw = bf && s.K % 8 == 0;
    *in_gy = bf && s.N % 8 == 0 && s.act == kActNone;
}

size_t linear_tc_workspace(const LinearShape& s, int bf, bool backward) {
    return backward ? plan_backward(s, bf).total : plan_forward(s, bf).total;
}

cudaError_t linear_tc_forward(const LinearShape& s, int bf, const void* x, const void* w, const void* bias,
                              const void* residual, void* y, void* z, void* ws, unsigned* status, cudaStream_t st,
                              int* launches) {
    if (bf)
        return forward_t(s, (const bf16*)x, (const bf16*)w, (const bf16*)bias, (const bf16*)residual, (bf16*)y,
                         (bf16*)z, (uint8_t*)ws, status, st, launches);
    return forward_t(s, (const float*)x, (const float*)w, (const float*)bias, (const float*)residual, (float*)y,
                     (float*)z, (uint8_t*)ws, status, st, launches);
}

cudaError_t linear_tc_backward(const LinearShape& s, int bf, const void* x, const void* w, const void* saved,
                               const void* gy, void* gx, float* gw, float* gb, void* gr, void* ws, unsigned* status,
                               cudaStream_t st, int* launches) {
    if (bf)
        return backward_t(s, (const bf16*)x, (const bf16*)w, (const bf16*)saved, (const bf16*)gy, (bf16*)gx, gw, gb,
                          (bf16*)gr, (uint8_t*)ws, status, st, launches);
    return backward_t(s, (const float*)x, (const float*)w, (const float*)saved, (const float*)gy, (float*)gx, gw, gb,
                      (float*)gr, (uint8_t*)ws, status, st, launches);
}

}  // namespace dcn
