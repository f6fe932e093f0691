// Linear layer (1x1 convolution of an NHWC map) on CUDA cores, for every size,
// type and alignment:
//   forward   z = x W^T + bias + residual, y = act(z)        x [M, K], W [N, K]
//   backward  dz = grad_y act'(s), grad_x = dz W, grad_W = dz^T x,
//             grad_bias = sum_m dz, grad_residual = dz
// One kernel computes a matrix product C[i, j] = sum_r A(i, r) B(r, j) over
// 64 x 64 tiles; A and B are read through functors, so dz is formed as it is
// loaded and no intermediate is stored. Sums are float32, in a fixed order.
#include <type_traits>

#include "act.cuh"
#include "kernels.h"

namespace dcn {
namespace {

constexpr int TILE = 64, DEPTH = 16, NT = 256;  // tile side, reduction step, threads (4 x 4 outputs each)

template <typename T>
struct Plain {  // element (i, r) of a matrix, or of its transpose
    const T* p;
    long long si, sr;
    __device__ float operator()(long long i, long long r) const { return ld1(p + i * si + r * sr); }
};

template <typename T, int ACT>
struct Dz {  // dz(i, r), or transposed
    const T *gy, *saved;
    long long si, sr;
    __device__ float operator()(long long i, long long r) const {
        const long long at = i * si + r * sr;
        const float g = ld1(gy + at);
        if constexpr (ACT == kActNone) return g;
        return act_grad<ACT, false>(g, ld1(saved + at));
    }
};

template <typename T, int ACT>
struct Epilogue {  // bias, residual, pre-activation, activation
    const T *bias, *residual;
    T *y, *z;
    long long ld;
    __device__ void operator()(long long i, long long j, float v) const {
        const long long at = i * ld + j;
        if (bias) v += ld1(bias + j);
        if (residual) v += ld1(residual + at);
        if (z) z[at] = from_float<T>(v);
        y[at] = from_float<T>(act_apply<ACT, false>(v));
    }
};

template <typename T>
struct Store {
    T* p;
    long long ld;
    __device__ void operator()(long long i, long long j, float v) const { p[i * ld + j] = from_float<T>(v); }
};

// C[i, j] for a 64 x 64 tile. AR / BR: consecutive threads walk the reduction
// index when loading A / B (its elements lie side by side in memory), else the
// row or column index.
template <bool AR, bool BR, typename FA, typename FB, typename FE>
__global__ void __launch_bounds__(NT) gemm_kernel(FA fa, FB fb, FE fe, long long I, long long J, long long R, int jt) {
    __shared__ float as[DEPTH][TILE + 1], bs[DEPTH][TILE + 1];
    const long long i0 = (long long)(blockIdx.x / jt) * TILE, j0 = (long long)(blockIdx.x % jt) * TILE;
    const int t = threadIdx.x, ti = t / 16, tj = t % 16;
    float acc[4][4] = {};
    for (long long r0 = 0; r0 < R; r0 += DEPTH) {
#pragma unroll
        for (int q = 0; q < TILE * DEPTH / NT; ++q) {
            const int e = t + q * NT;
            const int ar = AR ? e % DEPTH : e / TILE, ai = AR ? e / DEPTH : e % TILE;
            const int br = BR ? e % DEPTH : e / TILE, bj = BR ? e / DEPTH : e % TILE;
            as[ar][ai] = (i0 + ai < I && r0 + ar < R) ? fa(i0 + ai, r0 + ar) : 0.f;
            bs[br][bj] = (j0 + bj < J && r0 + br < R) ? fb(r0 + br, j0 + bj) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < DEPTH; ++r) {
            float a[4], b[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                a[q] = as[r][ti * 4 + q];
                b[q] = bs[r][tj * 4 + q];
            }
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[p][q] = fmaf(a[p], b[q], acc[p][q]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const long long i = i0 + ti * 4 + p, j = j0 + tj * 4 + q;
            if (i < I && j < J) fe(i, j, acc[p][q]);
        }
}

template <bool AR, bool BR, typename FA, typename FB, typename FE>
cudaError_t gemm(const FA& fa, const FB& fb, const FE& fe, long long I, long long J, long long R, cudaStream_t st) {
    const long long it = (I + TILE - 1) / TILE, jt = (J + TILE - 1) / TILE;
    if (it * jt >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    gemm_kernel<AR, BR><<<(unsigned)(it * jt), NT, 0, st>>>(fa, fb, fe, I, J, R, (int)jt);
    return cudaGetLastError();
}

// grad_bias[n] = sum_m dz[m, n]: 32 columns and 8 row lanes a block. Each lane
// adds its rows in runs of 64, so that no float32 chain grows with M.
template <typename F>
__global__ void __launch_bounds__(256) column_sum_kernel(F f, float* __restrict__ out, long long M, int N) {
    __shared__ float s[8][33];
    const int c = threadIdx.x % 32, l = threadIdx.x / 32;
    const long long n = (long long)blockIdx.x * 32 + c;
    double total = 0.0;
    if (n < N)
        for (long long m0 = l; m0 < M; m0 += 8 * 64) {
            float run = 0.f;
            for (int q = 0; q < 64 && m0 + 8 * q < M; ++q) run += f(m0 + 8 * q, n);
            total += run;
        }
    s[l][c] = (float)total;
    __syncthreads();
    if (l == 0 && n < N) {
        float v = 0.f;
        for (int q = 0; q < 8; ++q) v += s[q][c];
        out[n] = v;
    }
}

// grad_residual[m, n] = dz[m, n]
template <typename T, typename F>
__global__ void __launch_bounds__(256) dz_kernel(F f, T* __restrict__ out, long long M, int N) {
    const long long n = M * N;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL)
        out[i] = from_float<T>(f(0, i));
}

template <typename T>
cudaError_t forward_t(const LinearShape& s, const T* x, const T* w, const T* bias, const T* residual, T* y, T* z,
                      cudaStream_t st) {
    return with_act(s.act, [&](auto A) {
        return gemm<true, true>(Plain<T>{x, s.K, 1}, Plain<T>{w, 1, s.K},
                                Epilogue<T, decltype(A)::value>{bias, residual, y, z, s.N}, s.M, s.N, s.K, st);
    });
}

template <typename T>
cudaError_t backward_t(const LinearShape& s, const T* x, const T* w, const T* saved, const T* gy, T* gx, float* gw,
                       float* gb, T* gr, cudaStream_t st, int* launches) {
    return with_act(s.act, [&](auto A) {
        constexpr int ACT = decltype(A)::value;
        cudaError_t e = cudaSuccess;
        if (gr) {
            const long long n = ((long long)s.M * s.N + 255) / 256;
            dz_kernel<T><<<(unsigned)(n < 148 * 32 ? n : 148 * 32), 256, 0, st>>>(Dz<T, ACT>{gy, saved, 0, 1}, gr, s.M,
                                                                                 s.N);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
            ++*launches;
        }
        if (gx) {
            e = gemm<true, false>(Dz<T, ACT>{gy, saved, s.N, 1}, Plain<T>{w, s.K, 1}, Store<T>{gx, s.K}, s.M, s.K, s.N,
                                  st);
            if (e != cudaSuccess) return e;
            ++*launches;
        }
        if (gw) {
            e = gemm<false, false>(Dz<T, ACT>{gy, saved, 1, s.N}, Plain<T>{x, s.K, 1}, Store<float>{gw, s.K}, s.N, s.K,
                                   s.M, st);
            if (e != cudaSuccess) return e;
            ++*launches;
        }
        if (gb) {
            column_sum_kernel<<<(unsigned)((s.N + 31) / 32), 256, 0, st>>>(Dz<T, ACT>{gy, saved, s.N, 1}, gb, s.M, s.N);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
            ++*launches;
        }
        return e;
    });
}

}  // namespace

cudaError_t linear_forward(const LinearShape& s, int bf, const void* x, const void* w, const void* bias,
                           const void* residual, void* y, void* z, cudaStream_t st, int* launches) {
    ++*launches;
    if (bf)
        return forward_t(s, (const bf16*)x, (const bf16*)w, (const bf16*)bias, (const bf16*)residual, (bf16*)y,
                         (bf16*)z, st);
    return forward_t(s, (const float*)x, (const float*)w, (const float*)bias, (const float*)residual, (float*)y,
                     (float*)z, st);
}

cudaError_t linear_backward(const LinearShape& s, int bf, const void* x, const void* w, const void* saved,
                            const void* gy, void* gx, float* gw, float* gb, void* gr, cudaStream_t st, int* launches) {
    if (bf)
        return backward_t(s, (const bf16*)x, (const bf16*)w, (const bf16*)saved, (const bf16*)gy, (bf16*)gx, gw, gb,
                          (bf16*)gr, st, launches);
    return backward_t(s, (const float*)x, (const float*)w, (const float*)saved, (const float*)gy, (float*)gx, gw, gb,
                      (float*)gr, st, launches);
}

}  // namespace dcn
