// selective_scan.hpp -- what the selective scan's forward and backward share.
//
// Layout.  A wave holds a tile of 4 S states x 16 C channels: lane l owns
// channel pair (or channel) cl = l & 15 and states S sg ... S sg + S - 1,
// sg = l >> 4.  Sums over states are S in-lane terms joined over the four
// sixteen-lane rows (sg_join); rows of u, delta, z are read C channels a lane,
// row sg, sg + 4, ... of the wave's steps, so each value is read, passed
// through softplus and gated by one lane only, and the joined sums land on the
// lane that needs them.
//
// Time.  A workgroup walks the sequence of one channel tile in blocks of NW L
// steps; wave w scans steps [w L, (w + 1) L) of the block from a zero state,
// the per-wave transforms (P, S) meet in LDS, where the carries are folded, and
// every wave corrects its results with its carry.  Gates a = exp(dl A) are
// computed once and kept in registers for the correction.
#pragma once

#include "block_ops.hpp"

namespace miscan {

struct ScanArgs {
    const void *u, *delta, *z, *Bm, *Cm;
    const float *A, *skip, *delta_bias;
    const float *h0;       // forward
    const int32_t *lengths;
    void *y;
    float *hT;
    float *states;         // block states: written by the forward, read by the backward
    const void *dy;        // backward
    const float *dhT;
    void *du, *ddelta, *dz;
    float *dh0;
    float *part_bc;        // (tiles a group, 2, B, T, G, N) partial dBm, dCm
    float *part_a;         // (B, N + 2, D) partial dA (transposed), dskip, ddelta_bias
    int64_t B, T, D, N;
    int G, per;            // groups, channels a group
    int tiles;             // channel tiles a group
    int n_items;           // B * G * tiles
    int softplus;
    int vec;               // rows may be read C channels at a time
};

// Tile constants of a state count: S states a lane; C channels a lane and L
// steps a wave follow from a budget of 64 gates a lane (128 vector registers
// for gates and products in the backward).
template <int S> struct ScanTile;
template <> struct ScanTile<1> { static constexpr int C = 2, L = 16; };
template <> struct ScanTile<2> { static constexpr int C = 2, L = 16; };
template <> struct ScanTile<4> { static constexpr int C = 2, L = 8; };
template <> struct ScanTile<8> { static constexpr int C = 1, L = 8; };
template <> struct ScanTile<16> { static constexpr int C = 1, L = 4; };

constexpr int SCAN_NW = 8;  // waves a workgroup

inline int scan_s(int64_t N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

// Steps between two saved states: a block of the backward.
inline int64_t scan_block(int64_t N) {
    switch (scan_s(N)) {
        case 1: return SCAN_NW * ScanTile<1>::L;
        case 2: return SCAN_NW * ScanTile<2>::L;
        case 4: return SCAN_NW * ScanTile<4>::L;
        case 8: return SCAN_NW * ScanTile<8>::L;
    }
    return SCAN_NW * ScanTile<16>::L;
}

template <int S>
__host__ __device__ constexpr int64_t scan_block_of() { return SCAN_NW * ScanTile<S>::L; }

struct ScanSizes {
    int64_t x, bc, h, a, d, states;  // bytes of (B,T,D), Bm, (B,D,N), A, (D), states
};
mi_status check_scan(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, mi_dtype dt, ScanSizes *s);
bool scan_vec(const ScanArgs &a, mi_dtype dt);

// Work item of a workgroup.  Workgroups go to the 8 XCDs in turn; giving each
// XCD a consecutive run of items puts neighbouring channel tiles, which share
// 128-byte lines of every row, behind one L2.
__device__ __forceinline__ int xcd_item(int n) {
    const int per = (n + 7) / 8;
    return (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
}
inline unsigned xcd_grid(int n) { return (unsigned)((n + 7) / 8 * 8); }

// Row-joined sums: y[t][c] holds this lane's part for steps t = 4 j + i; on
// return out[j][c] is the sum over the four lane rows for step 4 j + sg.
// v_permlane32_swap / v_permlane16_swap exchange the halves (the odd and even
// rows) of two registers, so each exchange adds two steps at once.
__device__ __forceinline__ float swap_add32(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap_add16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
template <int L, int C>
__device__ __forceinline__ void sg_join(const float (&y)[L][C], float (&out)[L / 4][C]) {
#pragma unroll
    for (int j = 0; j < L / 4; ++j)
#pragma unroll
        for (int c = 0; c < C; ++c)
            out[j][c] = swap_add16(swap_add32(y[4 * j][c], y[4 * j + 2][c]),
                                   swap_add32(y[4 * j + 1][c], y[4 * j + 3][c]));
}

// C consecutive channels of a row; nv of them exist (0: none).  Missing ones
// are zero.
template <typename T, int C>
__device__ __forceinline__ void load_ch(const T *p, int nv, bool vec, float (&f)[C]) {
#pragma unroll
    for (int c = 0; c < C; ++c) f[c] = 0.f;
    if (nv == C && vec) {
        Pack<T, C>::unpack(load_vec<T, C>(p), f);
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (c < nv) f[c] = ld1(p + c);
    }
}
template <typename T, int C>
__device__ __forceinline__ void store_ch(T *p, int nv, bool vec, const float (&f)[C]) {
    if (nv == C && vec) {
        *reinterpret_cast<typename Pack<T, C>::raw_t *>(p) = Pack<T, C>::pack(f);
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (c < nv) st1(p + c, f[c]);
    }
}

// dl = softplus(raw) or raw, with its derivative.
__device__ __forceinline__ float gate_rate(float raw, int use_softplus, float *deriv) {
    float sig;
    const float sp = softplus(raw, &sig);
    *deriv = use_softplus ? sig : 1.f;
    return use_softplus ? sp : raw;
}

// Wave-level LDS ordering: data exchanged inside one wave needs its own LDS
// operations done, no workgroup barrier.
__device__ __forceinline__ void wave_lds_fence() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// N consecutive floats of LDS as 16-, 8- or 4-byte accesses.
template <int N>
__device__ __forceinline__ void lds_read(const float *p, float (&f)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const f32x4 q = *reinterpret_cast<const f32x4 *>(p + i);
            f[i] = q.x; f[i + 1] = q.y; f[i + 2] = q.z; f[i + 3] = q.w;
        }
    } else if constexpr (N == 2) {
        const f32x2 q = *reinterpret_cast<const f32x2 *>(p);
        f[0] = q.x; f[1] = q.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = p[i];
    }
}

// Per-lane vectors of EL floats in LDS, in groups of V = min(4, EL): element
// group g of lane l is at (g 64 + l) V, so a wave's accesses are consecutive.
template <int EL>
struct LaneVec {
    static constexpr int V = EL < 4 ? EL : 4;
    static __device__ __forceinline__ void write(float *p, int lane, const float (&f)[EL]) {
#pragma unroll
        for (int g = 0; g < EL / V; ++g) {
            float *q = p + (g * 64 + lane) * V;
            if constexpr (V == 4) *reinterpret_cast<f32x4 *>(q) = f32x4{f[4 * g], f[4 * g + 1], f[4 * g + 2], f[4 * g + 3]};
            else *reinterpret_cast<f32x2 *>(q) = f32x2{f[2 * g], f[2 * g + 1]};
        }
    }
    static __device__ __forceinline__ void read(const float *p, int lane, float (&f)[EL]) {
#pragma unroll
        for (int g = 0; g < EL / V; ++g) {
            const float *q = p + (g * 64 + lane) * V;
            if constexpr (V == 4) {
                const f32x4 r = *reinterpret_cast<const f32x4 *>(q);
                f[4 * g] = r.x; f[4 * g + 1] = r.y; f[4 * g + 2] = r.z; f[4 * g + 3] = r.w;
            } else {
                const f32x2 r = *reinterpret_cast<const f32x2 *>(q);
                f[2 * g] = r.x; f[2 * g + 1] = r.y;
            }
        }
    }
    // (lane, element) of linear position i
    static __device__ __forceinline__ void where(int i, int *lane, int *e) {
        *e = i / (64 * V) * V + i % V;
        *lane = i / V % 64;
    }
};

}  // namespace miscan
