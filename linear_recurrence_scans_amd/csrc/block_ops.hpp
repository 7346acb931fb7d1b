// block_ops.hpp -- device helpers shared by the block operators (causal
// convolution, selective scan, group norm): one-element IO, the activations
// and the fixed-order sum over partial results.
#pragma once

#include "common.hpp"

namespace miscan {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

template <typename T>
__device__ __forceinline__ float ld1(const T *p) {
    float f;
    Pack<T, 1>::unpack(*reinterpret_cast<const typename Pack<T, 1>::raw_t *>(p), &f);
    return f;
}
template <typename T>
__device__ __forceinline__ void st1(T *p, float f) {
    *reinterpret_cast<typename Pack<T, 1>::raw_t *>(p) = Pack<T, 1>::pack(&f);
}

// exp(x) as exp2 of the rounded product: its relative error grows as |x| 2^-24.
// sigmoid needs no more: far below zero its value is small in absolute terms, far
// above exp(-x) is small next to 1.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * LOG2E); }
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + fast_exp(-x)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
// d silu / dx from x and g = sigmoid(x)
__device__ __forceinline__ float dsilu(float x, float g) { return g * fmaf(x, 1.f - g, 1.f); }

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|), with a relative error below
// (8 + 0.05 |x|) 2^-24 where the result is small too (x far below zero, where e is all
// of it).  With p = -|x| log2(e) rounded, e = exp2(p) (1 + r), r = -|x| - p ln 2.  The
// logarithm of u = 1 + e lacks the rounding of u, e - (u - 1), and e r; both times 1 / u,
// which is near one where they count.  r of an infinite x is NaN and taken as -1, times e = 0.
// *sig receives sigmoid(x), the derivative, where it is wanted, as accurate.
__device__ __forceinline__ float softplus(float x, float *sig) {
    const float p = -fabsf(x) * LOG2E;
    const float e = __builtin_amdgcn_exp2f(p);
    const float u = 1.f + e;
    const float r = fmaxf(fmaf(p, -LN2, -fabsf(x)), -1.f);
    const float l = fmaf(__builtin_amdgcn_logf(u), LN2, fmaf(e, r, e - (u - 1.f)));
    if (sig != nullptr) {
        const float v = __builtin_amdgcn_rcpf(u);
        *sig = x >= 0.f ? v : fmaf(e, r, e) * v;
    }
    return fmaxf(x, 0.f) + l;
}

// The length of sequence b: lengths[b] clamped to [0, T], or T.
__device__ __forceinline__ int64_t seq_len(const int32_t *lengths, int64_t b, int64_t T) {
    if (lengths == nullptr) return T;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n > T ? T : n;
}

// Sum of P partial rows of M floats, handed to st(m, sum): 64 columns a
// workgroup, four threads a column that each add every fourth row, joined in a
// fixed order.  Reads each partial once with 256-byte rows.
template <class Store>
struct ReduceJob {
    const float *part;
    int64_t P, M;
    Store st;
    int blocks;  // workgroups of this job
};
constexpr int64_t REDUCE_BLOCKS = 16384;

template <class Store>
__device__ __forceinline__ void reduce_job(const ReduceJob<Store> &j, int block) {
    __shared__ float acc[4][64];
    const int col = threadIdx.x & 63, row = threadIdx.x >> 6;
    for (int64_t m0 = (int64_t)block * 64; m0 < j.M; m0 += (int64_t)j.blocks * 64) {
        const int64_t m = m0 + col;
        float s = 0.f;
        if (m < j.M) {
            const float *q = j.part + m;
#pragma unroll 4
            for (int64_t p = row; p < j.P; p += 4) s += q[p * j.M];
        }
        acc[row][col] = s;
        __syncthreads();
        if (row == 0 && m < j.M) j.st(m, (acc[0][col] + acc[1][col]) + (acc[2][col] + acc[3][col]));
        __syncthreads();
    }
}
template <class Store>
__global__ __launch_bounds__(256) void reduce_parts_kernel(ReduceJob<Store> j) {
    reduce_job(j, (int)blockIdx.x);
}
// Two sums in one launch.
template <class S1, class S2>
__global__ __launch_bounds__(256) void reduce_two_kernel(ReduceJob<S1> a, ReduceJob<S2> b) {
    if ((int)blockIdx.x < a.blocks) reduce_job(a, (int)blockIdx.x);
    else reduce_job(b, (int)blockIdx.x - a.blocks);
}

template <class Store>
inline ReduceJob<Store> reduce_of(const float *part, int64_t P, int64_t M, Store st) {
    const int64_t blocks = (M + 63) / 64;
    return {part, P, M, st, (int)(blocks < REDUCE_BLOCKS ? blocks : REDUCE_BLOCKS)};
}
template <class Store>
inline mi_status reduce_parts(const float *part, int64_t P, int64_t M, Store st, hipStream_t s) {
    const ReduceJob<Store> j = reduce_of(part, P, M, st);
    if (j.blocks == 0) return MI_OK;
    hipLaunchKernelGGL(reduce_parts_kernel<Store>, dim3((unsigned)j.blocks), dim3(256), 0, s, j);
    return launch_status();
}

}  // namespace miscan
