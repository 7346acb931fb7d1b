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
// Few channels.  Where the channel tiles do not fill the GPU, the sequence is cut
// into segments with a workgroup each: a first kernel forms every segment's
// transform (gates' product P, scan from zero), and a workgroup of the second
// folds those before (in the backward: after) its own, in order, to what enters
// its segment.  The gates are then formed twice, 17 issue slots a state-step
// instead of 12, on as many CUs as there are.
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
    float *part_a;         // (B * n_seg, N + 2, D) partial dA (transposed), dskip, ddelta_bias
    int64_t B, T, D, N;
    int G, per;            // groups, channels a group
    int tiles;             // channel tiles a group
    int n_seg;             // segments of the sequence, one workgroup each
    int64_t seg;           // steps a segment: whole blocks
    float *seg_v, *seg_p;  // (n_seg, B, D, N) transform of a segment: its scan from zero, the root of its gates' product
    int n_items;           // n_seg * B * G * tiles
    int softplus;
    int vec;               // rows may be read two channels at a time: no tile ends inside a pair
};

// Tiles by S, the states a lane holds: C channels a lane, L steps a wave, NW waves
// a workgroup.  S C L is the gates a lane keeps: 64, or 32 for S = 1 and 2, whose
// rows fill the LDS first.  A block of the backward, NW L steps, is also the
// distance of the states that the forward saves for it.  (The backward with 32
// gates and 16 waves a workgroup, four a SIMD, is slower at N = 16: 630 us against
// 535 for B = 4, T = 4096, D = 2048; its folds are twice as many and twice as long.)
template <int S> struct FwdTile;
template <> struct FwdTile<1> { static constexpr int C = 2, L = 16; };
template <> struct FwdTile<2> { static constexpr int C = 2, L = 8; };
template <> struct FwdTile<4> { static constexpr int C = 2, L = 8; };
template <> struct FwdTile<8> { static constexpr int C = 1, L = 8; };
template <> struct FwdTile<16> { static constexpr int C = 1, L = 4; };
template <int S> struct BwdTile : FwdTile<S> { static constexpr int NW = 8; };

// Rows inside a block are addressed with 32-bit byte offsets: 16 rows of D
// (or G N) 4-byte values stay below 2^31.
constexpr int64_t SCAN_MAX_D = 1 << 24;

inline int scan_s(int64_t N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

// Steps between two saved states.
template <int S>
__host__ __device__ constexpr int64_t scan_block_of() { return BwdTile<S>::NW * BwdTile<S>::L; }
inline int64_t scan_block(int64_t N) {
    switch (scan_s(N)) {
        case 1: return scan_block_of<1>();
        case 2: return scan_block_of<2>();
        case 4: return scan_block_of<4>();
        case 8: return scan_block_of<8>();
    }
    return scan_block_of<16>();
}

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
// Sequences vary fastest, so that short and long ones spread over the XCDs.
struct Item {
    int b, tile, g, seg;
    __device__ __forceinline__ Item(int item, const ScanArgs &p) {
        const int nb = (int)p.B;
        b = item % nb;
        tile = item / nb % p.tiles;
        g = item / nb / p.tiles % p.G;
        seg = item / nb / p.tiles / p.G;
    }
};
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
// Joins four consecutive steps.
template <int C>
__device__ __forceinline__ void sg_join4(const float (&y0)[C], const float (&y1)[C], const float (&y2)[C],
                                         const float (&y3)[C], float (&out)[C]) {
#pragma unroll
    for (int c = 0; c < C; ++c) out[c] = swap_add16(swap_add32(y0[c], y2[c]), swap_add32(y1[c], y3[c]));
}
template <int L, int C>
__device__ __forceinline__ void sg_join(const float (&y)[L][C], float (&out)[L / 4][C]) {
#pragma unroll
    for (int j = 0; j < L / 4; ++j) sg_join4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3], out[j]);
}

// Row access.  A wave's block of rows is one buffer descriptor whose size ends
// after the last step that exists, so a lane needs 32-bit offsets only, and
// steps past a sequence's end read as zero without a select; so do channels past
// the tile's end, whose offset is NO_CHANNEL.  Rows are read with the default
// cache policy: a 128-byte line holds the channels of two to four tiles.
constexpr uint32_t NO_CHANNEL = 0x7ffffff0u;

template <typename T, int N>
__device__ __forceinline__ typename Pack<T, N>::raw_t buf_read(rsrc_t r, uint32_t voff) {
    using raw_t = typename Pack<T, N>::raw_t;
    constexpr int BYTES = (int)sizeof(T) * N;
    if constexpr (BYTES == 8) return __builtin_bit_cast(raw_t, __builtin_amdgcn_raw_buffer_load_b64(r, voff, 0, 0));
    else if constexpr (BYTES == 4) return __builtin_bit_cast(raw_t, __builtin_amdgcn_raw_buffer_load_b32(r, voff, 0, 0));
    else return __builtin_bit_cast(raw_t, __builtin_amdgcn_raw_buffer_load_b16(r, voff, 0, 0));
}

// Products of gates.  Rates of growth (A > 0, or negative rates without softplus)
// can take the product P of a run of gates past fp32's range where the state that
// it multiplies is zero or small and the result is finite: inf 0 would be NaN.  P
// is therefore held as its square root, at most 2^127, and applied twice, which
// covers whatever a normal state and its result can span.  (A NaN in P is one in
// the run's scan from zero too.)  The forward's blocks use P itself and redo a fold
// that ends in no finite value step by step: for B = 8, T = 4096, D = 4096, N = 16, bf16
// that costs 2 to 5 us of 740, roots 21; the backward has no registers for it (50 us of
// 726 for B = 4, T = 4096, D = 2048 with its forward, roots 6).
__device__ __forceinline__ float root_product(float e) {  // e: log2 of the product
    return __builtin_amdgcn_exp2f(fminf(0.5f * e, 127.f));
}
__device__ __forceinline__ float carry_through(float root, float carry, float s) { return fmaf(root, root * carry, s); }
__device__ __forceinline__ float join_roots(float a, float b) { return fminf(a * b, 0x1p127f); }

// The C channels of J rows at offsets voff: whole vectors (a lane then has C
// channels or none), or single elements of which the first nv exist.
template <typename T, int C, int J>
__device__ __forceinline__ void load_rows(rsrc_t r, const uint32_t (&voff)[J], int nv, bool whole,
                                          typename Pack<T, C>::raw_t (&raw)[J]) {
    if (whole) {
#pragma unroll
        for (int j = 0; j < J; ++j) raw[j] = buf_read<T, C>(r, voff[j]);
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float f[C];
#pragma unroll
            for (int c = 0; c < C; ++c)
                Pack<T, 1>::unpack(buf_read<T, 1>(r, c < nv ? voff[j] + c * (uint32_t)sizeof(T) : NO_CHANNEL), f + c);
            raw[j] = Pack<T, C>::pack(f);
        }
    }
}

// The C channels of a lane's row, of which the first nv exist.
template <typename T, int C>
__device__ __forceinline__ void store_ch(char *p, int nv, bool whole, const float (&f)[C]) {
    if (whole) {
        if (nv > 0) *reinterpret_cast<typename Pack<T, C>::raw_t *>(p) = Pack<T, C>::pack(f);
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (c < nv) st1(reinterpret_cast<T *>(p) + c, f[c]);
    }
}

// Steps of [t0, t0 + L) before `end`.
template <int L>
__device__ __forceinline__ int steps_left(int64_t t0, int64_t end) {
    return t0 >= end ? 0 : end - t0 < L ? (int)(end - t0) : L;
}

// dl = softplus(raw) or raw, with its derivative where `deriv` is not null.
__device__ __forceinline__ float gate_rate(float raw, int use_softplus, float *deriv) {
    if (use_softplus) return softplus(raw, deriv);
    if (deriv != nullptr) *deriv = 1.f;
    return raw;
}

// A log2(e), the factor of a gate's exponent.  It is kept finite (a NaN stays one), so
// that a rate of zero, which is also what a step that does not exist has, makes a gate
// of one for A = -inf too.
__device__ __forceinline__ float gate_base(float A) {
    const float a = A * LOG2E;
    return a < -__FLT_MAX__ ? -__FLT_MAX__ : a;
}

// LDS ordering.  Fences of the local address space make the compiler and the
// LDS queue keep the order without waiting for global loads in flight, which a
// __syncthreads() would drain.  wave_lds_sync: data exchanged inside one wave;
// wg_lds_sync: inside the workgroup.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}
__device__ __forceinline__ void wg_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Bm rows.  All lanes of a quad need the same S values of a row (their states'),
// so a lane holds every fourth only: register i of lane l is state 4 i + (l & 3)
// of its S (l & 1 for S = 2), and a multiplication takes state s from its quad
// with a DPP operand, at no extra instruction.  Held as [state][step] in LDS,
// four steps come with one 16-byte read.  (fma has no DPP form here, so Cm rows
// are read whole.)
template <int S>
struct QuadRow {
    static constexpr int NB = (S + 3) / 4, MASK = S >= 4 ? 3 : S - 1;
    static __device__ __forceinline__ int first(int lane) { return (lane >> 4) * S + (lane & MASK); }
    template <int s>
    static __device__ __forceinline__ float get(const float (&r)[NB]) {
        constexpr int q = s & 3;
        if constexpr (S == 1) return r[0];
        else return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, r[s / 4]), q * 0x55, 0xf,
                                                                       0xf, true));
    }
};

// for_each<N>(f): f(Num<0>()), ..., f(Num<N - 1>()): loops whose index is a
// constant expression.
template <int K> struct Num { static constexpr int value = K; };
template <int N, int I = 0, class F>
__device__ __forceinline__ void for_each(F &&f) {
    if constexpr (I < N) {
        f(Num<I>());
        for_each<N, I + 1>(f);
    }
}

// Pins C values to this point of the program: the compiler otherwise sinks sums
// that are needed later to their use and keeps all their terms in registers.
template <int C>
__device__ __forceinline__ void pin(float (&v)[C]) {
#pragma unroll
    for (int c = 0; c < C; ++c) asm volatile("" : "+v"(v[c]));
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

// N consecutive floats of a lane's own.
template <int N>
__device__ __forceinline__ void lds_write(float *p, const float (&f)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<f32x4 *>(p + i) = f32x4{f[i], f[i + 1], f[i + 2], f[i + 3]};
    } else if constexpr (N == 2) {
        *reinterpret_cast<f32x2 *>(p) = f32x2{f[0], f[1]};
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = f[i];
    }
}

// Per-lane vectors of EL floats in LDS, in groups of V = min(4, EL): element
// group g of lane l is at (g 64 + l) V, so a wave's accesses are consecutive.
template <int EL>
struct LaneVec {
    static constexpr int V = EL < 4 ? EL : 4;
    static_assert(V == 1 || V == 2 || V == 4, "elements a lane");
    static __device__ __forceinline__ void write(float *p, int lane, const float (&f)[EL]) {
#pragma unroll
        for (int g = 0; g < EL / V; ++g) {
            float *q = p + (g * 64 + lane) * V;
            if constexpr (V == 4) *reinterpret_cast<f32x4 *>(q) = f32x4{f[4 * g], f[4 * g + 1], f[4 * g + 2], f[4 * g + 3]};
            else if constexpr (V == 2) *reinterpret_cast<f32x2 *>(q) = f32x2{f[2 * g], f[2 * g + 1]};
            else *q = f[g];
        }
    }
    static __device__ __forceinline__ void read(const float *p, int lane, float (&f)[EL]) {
#pragma unroll
        for (int g = 0; g < EL / V; ++g) {
            float v[V];
            lds_read<V>(p + (g * 64 + lane) * V, v);
#pragma unroll
            for (int i = 0; i < V; ++i) f[g * V + i] = v[i];
        }
    }
    // (lane, element) of linear position i
    static __device__ __forceinline__ void where(int i, int *lane, int *e) {
        *e = i / (64 * V) * V + i % V;
        *lane = i / V % 64;
    }
};

}  // namespace miscan
