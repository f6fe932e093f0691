// The linear layer's forward for a few rows (M <= 8: the RoIs left in an image,
// one pixel), in one launch on CUDA cores: y = act(x W^T + bias + residual).
//
// Such a product reads the weight once and does next to nothing with it, so it is
// bound by the weight's bytes and by latency. A block's warps form teams of one to
// eight; a team takes a group of NR rows of W at a time and shares its reduction
// (each lane a 16-byte vector of every row at a time), so that its loads lie side by
// side, no part of a sum leaves the block, and x comes from L1 after the first group,
// for all teams. Sums are float32 pairs (fma.f32x2), joined by a butterfly over the
// lanes and then over the team's warps, in a fixed order.
//
// N x K of 1024 x 12544 bfloat16 (25.7 MB, 3.9 us at HBM rate): 6 to 7 us for one
// row, 8.5 for two, 11 to 12 for five, 13.6 for eight: the more rows, the more of the
// time goes to x's loads (two of the weight's rows for each of them) and the sums. The
// tensor-core kernel, with its reduction split 18 times and a joining launch, takes
// 13.5 us for nine. float32: 10.4 us for one row, 23 for eight, tensor cores 45.2.
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "kernels.h"
#include "norm.cuh"
#include "tc_ptx.cuh"

namespace dcn {
namespace {

constexpr int NT = 256, WARPS = NT / 32;

// Sum over the lanes of NV values each (NV a power of two up to 32); lane l returns the sum of value l % NV.
template <int NV>
__device__ __forceinline__ float butterfly(float (&v)[NV]) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int o = 16; o >= NV; o /= 2)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(~0u, v[i], o);
#pragma unroll
    for (int o = NV / 2, n = NV; o >= 1; o /= 2, n /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = up ? v[i + n / 2] : v[i], send = up ? v[i] : v[i + n / 2];
            v[i] = keep + __shfl_xor_sync(~0u, send, o);
        }
    }
    return v[0];
}

template <typename T, int NR, int MB, int ACT>
__global__ void __launch_bounds__(NT, MB > 2 ? 2 : 3)
    few_kernel(const T* __restrict__ x, const T* __restrict__ w, const T* __restrict__ bias, const T* residual, T* y, T* z,
               int M, int N, int K, int team) {
    constexpr int V = 16 / (int)sizeof(T), P = V / 2, DEPTH = 8 / NR;
    constexpr int MP = MB == 6 ? 8 : MB, NV = NR * MP;  // the butterfly wants a power of two
    __shared__ float sm[WARPS][NV];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, kv = K / V;
    // rows past the last read the last (their sums are dropped)
    const T* xp[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) xp[m] = x + (size_t)min(m, M - 1) * K;
    const int teams = WARPS / team, first = warp % team * 32 + lane, step = team * 32;
    for (int g = blockIdx.x * teams; g * NR < N; g += gridDim.x * teams) {
        const int n0 = (g + warp / team) * NR;
        const T* wp[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) wp[r] = w + (size_t)min(n0 + r, N - 1) * K;
        F2 acc[NR][MB] = {};
        for (int i0 = first; i0 < kv; i0 += DEPTH * step) {
            uint4 q[DEPTH][NR];  // the weight's loads first, all in flight
#pragma unroll
            for (int d = 0; d < DEPTH; ++d)
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if (d == 0 || i0 + d * step < kv) q[d][r] = ptx::ldg_v4_stream(wp[r] + (size_t)(i0 + d * step) * V);
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                const int i = i0 + d * step;
                if (d > 0 && i >= kv) break;
                F2 a[NR][P];
#pragma unroll
                for (int r = 0; r < NR; ++r) unpack(a[r], q[d][r]);
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    F2 b[P];
                    unpack(b, __ldg(reinterpret_cast<const uint4*>(xp[m] + (size_t)i * V)));
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int p = 0; p < P; ++p) acc[r][m] = fma(a[r][p], b[p], acc[r][m]);
                }
            }
        }
        float v[NV] = {};
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                float lo, hi;
                split(acc[r][m], lo, hi);
                v[r * MP + m] = lo + hi;
            }
        float sum = butterfly<NV>(v);
        if (team > 1) {
            if (lane < NV) sm[warp][lane] = sum;
            __syncthreads();
            if (warp % team == 0 && lane < NV)
                for (int k = 1; k < team; ++k) sum += sm[warp + k][lane];
            __syncthreads();  // sm is free
        }
        const int n = n0 + lane / MP, m = lane % MP;
        if (warp % team == 0 && lane < NV && n < N && m < M) {
            const size_t at = (size_t)m * N + n;
            if (bias) sum += ld1(bias + n);
            if (residual) sum += ld1(residual + at);
            if (z) z[at] = from_float<T>(sum);
            y[at] = from_float<T>(act_apply<ACT, kFast<T>>(sum));
        }
    }
}

template <typename T, int NR, int MB>
cudaError_t run(const LinearShape& s, const T* x, const T* w, const T* bias, const T* residual, T* y, T* z,
                cudaStream_t st) {
    return with_act(s.act, [&](auto A) {
        // Warps that share a group: with many rows of x few, so that a block's teams read the same x from L1 (5 x 1024
        // x 12544 bfloat16, eight warps 14.2 us, four 12.5), unless too few blocks are left (float32 5 x 2048 x 2048,
        // one warp 10.1 us, two 7.0).
        const int groups = (s.N + NR - 1) / NR, kv = s.K / (16 / (int)sizeof(T));
        int team = 1;
        while (team < WARPS &&
               (kv > team * (MB > 2 ? 512 : 64) || (kv > team * 256 && (long long)groups * team < WARPS * num_sms())))
            team *= 2;
        const int teams = WARPS / team;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)std::min((groups + teams - 1) / teams, num_sms() * (MB > 2 ? 2 : 3)));
        cfg.blockDim = dim3(NT);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, few_kernel<T, NR, MB, decltype(A)::value>, x, w, bias, residual, y, z, s.M, s.N,
                                  s.K, team);
    });
}

// Rows of W at a time: four where x takes few registers beside them, unless that leaves SMs without a block.
template <typename T, int MB>
cudaError_t run_m(const LinearShape& s, const T* x, const T* w, const T* bias, const T* residual, T* y, T* z,
                  cudaStream_t st) {
    if constexpr (MB <= 2)
        if (s.N >= 4 * 148) return run<T, 4, MB>(s, x, w, bias, residual, y, z, st);
    return run<T, 2, MB>(s, x, w, bias, residual, y, z, st);
}

template <typename T>
cudaError_t forward_t(const LinearShape& s, const T* x, const T* w, const T* bias, const T* residual, T* y, T* z,
                      cudaStream_t st) {
    if (s.M == 1) return run_m<T, 1>(s, x, w, bias, residual, y, z, st);
    if (s.M == 2) return run_m<T, 2>(s, x, w, bias, residual, y, z, st);
    if (s.M <= 4) return run_m<T, 4>(s, x, w, bias, residual, y, z, st);
    // (eight rows' kernel for five took 14.2 us where this one's 10.9 to 12)
    if (s.M <= 6) return run_m<T, 6>(s, x, w, bias, residual, y, z, st);
    return run_m<T, 8>(s, x, w, bias, residual, y, z, st);
}

}  // namespace

// More rows of a large bfloat16 weight keep the tensor cores, whose time hardly grows with them: 5 x 4096 x 4096 takes
// 13.0 us here and 12.6 there, 8 x 4096 x 4096 15.6 and 12.4, 4 x 2048 x 12544 16.1 and 16.9, 4 x 8192 x 4096 19.3 and
// 18.4; but 5 x 1024 x 12544 10.9 and 13.3, 2 x 4096 x 4096 10.5 and 12.6. (float32 5 x 4096 x 4096 19 and 56 us.)
bool linear_few_supported(const LinearShape& s, int bf) {
    if (s.M > 8 || s.K % (bf ? 8 : 4)) return false;
    return !bf || s.M <= 2 || (long long)s.N * s.K < (s.M <= 4 ? 1LL << 25 : 1LL << 24);
}

cudaError_t linear_few_forward(const LinearShape& s, int bf, const void* x, const void* w, const void* bias,
                               const void* residual, void* y, void* z, cudaStream_t st) {
    return bf ? forward_t(s, (const bf16*)x, (const bf16*)w, (const bf16*)bias, (const bf16*)residual, (bf16*)y,
                          (bf16*)z, st)
              : forward_t(s, (const float*)x, (const float*)w, (const float*)bias, (const float*)residual, (float*)y,
                          (float*)z, st);
}

}  // namespace dcn
