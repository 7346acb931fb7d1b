// selective_scan_bwd.hip -- gradient of the selective state-space scan.
//
// A workgroup walks the blocks of one channel tile in reverse, each from the
// state the forward saved before it.  Inside a block every wave scans its steps
// forward (states) and in reverse (g a) from zero, one meeting in LDS folds both
// carries, and every wave then runs its steps forward from its true state
// (keeping a_t h_{t-1}) and in reverse from its true g.  Per state-step: gate 3
// issue slots (mul, exp2), local scans 4, states 2 to 4, gradients 7.
//
// Measured (MI355X, N = 16, bf16, z): B = 4, T = 4096, D = 2048 493 us (256
// workgroups, one a CU) and 23 for the closing sums, 26 slots a state-step, the vector ALU
// busy for 73 % of it; the rest are the two meetings a block, and LDS latency that two
// waves a SIMD do not hide.  Forward and backward of that size in us, and the MB of partial
// sums: N = 4 460 (34), 8 555 (67), 16 731 (135), 32 1747 (538), 64 3402 (1076).
//
// dBm and dCm sum over the channels of a group: C of them in the lane, sixteen
// lanes through LDS, the tiles of a group through partial rows that
// reduce_parts adds in a fixed order.
#include <stddef.h>

#include "checks.hpp"
#include "selective_scan.hpp"

namespace miscan {
namespace {

// Steps joined over the channel lanes at once: 16 values a lane, so that the join
// leaves one sum to every lane.
constexpr int join_steps(int S, int L) { return 16 / S < L ? 16 / S : L; }

// LDS of a wave.  `join` holds the values to sum over the channel lanes (rows four
// banks apart); it takes the place of s and p, which are done with by then.
template <int S, int C, int L>
struct BwdWave {
    static constexpr int E = S * C * 64, TR = join_steps(S, L), V = TR * S, ROW = 4 * V + 4;
    float x[L][16][2 * C];       // dl, dl u
    float ds[L][16][C];
    float b[L][4 * S];           // Bm
    float c[L][4 * S];           // Cm
    union {
        struct { float s[E], p[E]; };
        float join[16][ROW];
    };
    float r[E];
    float keep[3][64][L / 4 * C];  // a lane's own u, softplus', dy silu'(z) from staging to the last rows
};

// One float of every wave's LDS.  An LDS access reaches 64 KiB past its address
// register, less than the waves' span, so a register serves a few waves; the
// asm keeps the compiler from a register for each.
template <class W, int NW>
struct WaveColumn {
    static constexpr int REACH = 65536 / (int)sizeof(W);
    float *base[(NW + REACH - 1) / REACH];
    __device__ __forceinline__ WaveColumn(char *smem, int off) {
#pragma unroll
        for (int g = 0; g < (NW + REACH - 1) / REACH; ++g) {
            int o = off + g * REACH * (int)sizeof(W);
            asm volatile("" : "+v"(o));
            base[g] = reinterpret_cast<float *>(smem + o);
        }
    }
    __device__ __forceinline__ float &operator[](int w) const {
        return base[w / REACH][w % REACH * (int)(sizeof(W) / 4)];
    }
};

// Sums the sixteen channel lanes' values of TR steps and stores them: linear
// value o of 4 V is (row o / V, step o % V / S, state o % S).
template <int S, int TR, int ROW, typename F>
__device__ __forceinline__ void join_channels(const float (*red)[ROW], int lane, F store) {
    constexpr int V = TR * S, PER = 4 * V / 64;
    float acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll
    for (int c = 0; c < 16; ++c)
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] += red[c][lane * PER + i];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int o = lane * PER + i;
        store(o % V / S, o / V * S + o % S, acc[i]);
    }
}

// The first kernel of a cut sequence: every segment's reverse transform, the
// gradient that leaves its left end for none entering at its right, and the
// product of its gates.
template <typename T, int S, int C, int L, int NW>
__global__ __launch_bounds__(NW * 64) void scan_bwd_sum_kernel(ScanArgs p) {
    constexpr int EL = S * C, J = L / 4, NP = 4 * S;
    constexpr int E = EL * 64, NT = NW * 64, FPT = (E + NT - 1) / NT, BPL = (L * NP + 63) / 64;
    using LV = LaneVec<EL>;
    using PC = Pack<T, C>;
    using raw_t = typename PC::raw_t;
    using one_t = typename Pack<T, 1>::raw_t;
    __shared__ __align__(16) float sm_x[NW][L][16][2 * C];  // dl, ds
    __shared__ __align__(16) float sm_c[NW][L][NP];
    __shared__ __align__(16) float sm_r[NW][E], sm_p[NW][E];
    const int item = xcd_item(p.n_items);
    if (item >= p.n_items) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int sg = lane >> 4, cl = lane & 15;
    const Item it(item, p);
    const int tile = it.tile, g = it.g, seg = it.seg + 1;  // nothing needs the first segment's
    const int64_t b = it.b;
    const int ch0 = tile * 16 * C;
    const int64_t d0 = (int64_t)g * p.per + ch0;
    const int nch = p.per - ch0 < 16 * C ? p.per - ch0 : 16 * C;
    const int nv = nch - cl * C < 0 ? 0 : nch - cl * C > C ? C : nch - cl * C;
    const int64_t len = seq_len(p.lengths, b, p.T);
    const bool whole = C == 1 || p.vec;
    float A2[S][C], bias[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t d = d0 + cl * C + c;
        bias[c] = c < nv && p.delta_bias ? p.delta_bias[d] : 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int n = sg * S + s;
            A2[s][c] = c < nv && n < p.N ? gate_base(p.A[d * p.N + n]) : 0.f;
        }
    }
    float edge[FPT], prod[FPT];
#pragma unroll
    for (int f = 0; f < FPT; ++f) {
        edge[f] = 0.f;
        prod[f] = 1.f;
    }
    const uint32_t row = (uint32_t)(p.D * (int64_t)sizeof(T));
    uint32_t voff[J], coff[BPL];
#pragma unroll
    for (int j = 0; j < J; ++j)
        voff[j] = nv > 0 ? (uint32_t)(4 * j + sg) * row + (uint32_t)(cl * C * sizeof(T)) : NO_CHANNEL;
    const int64_t row0 = b * p.T * p.D + d0;
    const int64_t brow = (int64_t)p.G * p.N, b0 = (b * p.T * p.G + g) * p.N;
#pragma unroll
    for (int i = 0; i < BPL; ++i) {
        const int q = lane + 64 * i, t = q / NP, n = q % NP;
        coff[i] = q < L * NP && n < p.N ? (uint32_t)((t * brow + n) * (int64_t)sizeof(T)) : NO_CHANNEL;
    }
    raw_t dr[J], zr[J], gr[J];
    one_t cr[BPL];
    const auto load = [&](int64_t t0) {
        const int64_t left = steps_left<L>(t0, len);
        load_rows<T, C, J>(make_rows(static_cast<const T *>(p.delta) + row0 + t0 * p.D, left * row), voff, nv, whole,
                           dr);
        load_rows<T, C, J>(make_rows(static_cast<const T *>(p.dy) + row0 + t0 * p.D, left * row), voff, nv, whole, gr);
        if (p.z)
            load_rows<T, C, J>(make_rows(static_cast<const T *>(p.z) + row0 + t0 * p.D, left * row), voff, nv, whole,
                               zr);
        const rsrc_t rc = make_rows(static_cast<const T *>(p.Cm) + b0 + t0 * brow, left * brow * (int64_t)sizeof(T));
#pragma unroll
        for (int i = 0; i < BPL; ++i) cr[i] = buf_read<T, 1>(rc, coff[i]);
    };
    const int64_t blk0 = seg * (p.seg / (NW * L));
    const int64_t end = blk0 + p.seg / (NW * L);
    // blocks past the sequence's end pass the gradient on
    const int64_t live = (len + NW * L - 1) / (NW * L), blk1 = end < live ? end : live;
    if (blk1 > blk0) load((blk1 - 1) * (NW * L) + wave * L);
    for (int64_t blk = blk1 - 1; blk >= blk0; --blk) {
        const int64_t t0 = blk * (NW * L) + wave * L;
        const int left = steps_left<L>(t0, len);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float dd[C], z[C], gy[C], x[2 * C];
            PC::unpack(dr[j], dd);
            PC::unpack(gr[j], gy);
            if (p.z) PC::unpack(zr[j], z);
            const bool in = 4 * j + sg < left;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float r = gate_rate(dd[c] + bias[c], p.softplus, nullptr);
                x[c] = in ? r : 0.f;
                x[C + c] = p.z ? gy[c] * silu(z[c]) : gy[c];
            }
            lds_write<2 * C>(sm_x[wave][4 * j + sg][cl], x);
        }
#pragma unroll
        for (int i = 0; i < BPL; ++i) {
            const int q = lane + 64 * i;
            if (L * NP % 64 == 0 || q < L * NP) Pack<T, 1>::unpack(cr[i], &sm_c[wave][q / NP][q % NP]);
        }
        if (blk > blk0) load(t0 - NW * L);
        wave_lds_sync();
        float gv[EL], pv[EL], sum[C];
#pragma unroll
        for (int c = 0; c < C; ++c) sum[c] = 0.f;
#pragma unroll
        for (int t = L - 1; t >= 0; --t) {
            float x[2 * C], ct[S];
            lds_read<2 * C>(sm_x[wave][t][cl], x);
            lds_read<S>(&sm_c[wave][t][sg * S], ct);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                sum[c] += x[c];
#pragma unroll
                for (int s = 0; s < S; ++s)
                    gv[c * S + s] = __builtin_amdgcn_exp2f(x[c] * A2[s][c]) *
                                    (t == L - 1 ? ct[s] * x[C + c] : fmaf(ct[s], x[C + c], gv[c * S + s]));
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int s = 0; s < S; ++s) pv[c * S + s] = root_product(sum[c] * A2[s][c]);
        LV::write(sm_r[wave], lane, gv);
        LV::write(sm_p[wave], lane, pv);
        wg_lds_sync();
#pragma unroll
        for (int f = 0; f < FPT; ++f) {
            const int i = tid + f * NT;
            if (i < E) {
#pragma unroll
                for (int w = NW - 1; w >= 0; --w) {
                    edge[f] = carry_through(sm_p[w][i], edge[f], sm_r[w][i]);
                    prod[f] = join_roots(prod[f], sm_p[w][i]);
                }
            }
        }
        wg_lds_sync();
    }
#pragma unroll
    for (int f = 0; f < FPT; ++f) {
        const int i = tid + f * NT;
        int ln, e;
        LV::where(i < E ? i : 0, &ln, &e);
        const int n = (ln >> 4) * S + e % S, ch = (ln & 15) * C + e / S;
        if (i < E && n < p.N && ch < nch) {
            const int64_t at = ((seg * p.B + b) * p.D + d0 + ch) * p.N + n;
            p.seg_v[at] = edge[f];
            p.seg_p[at] = prod[f];
        }
    }
}

template <typename T, int S, int C, int L, int NW, bool GATED>
__global__ __launch_bounds__(NW * 64, 2) void scan_bwd_kernel(ScanArgs p) {
    constexpr int EL = S * C, J = L / 4, NP = 4 * S;
    constexpr int E = EL * 64, NT = NW * 64, BPL = (L * NP + 63) / 64;
    constexpr int FPT = (2 * E + NT - 1) / NT;  // folds a thread: E forward, E in reverse
    using LV = LaneVec<EL>;
    using PC = Pack<T, C>;
    using raw_t = typename PC::raw_t;
    using one_t = typename Pack<T, 1>::raw_t;
    using W = BwdWave<S, C, L>;
    constexpr int TR = W::TR, V = W::V;
    // Gates and products a_t h_{t-1} both stay in registers, up to 128 of them;
    // with 16 states a lane the gates are formed again (3 of 28 issue slots).
    constexpr bool KEEP = S < 16;
    extern __shared__ __align__(16) char smem[];
    W *const sm = reinterpret_cast<W *>(smem);
    const int item = xcd_item(p.n_items);
    if (item >= p.n_items) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    W &my = sm[wave];
    const int sg = lane >> 4, cl = lane & 15;
    const Item it(item, p);
    const int tile = it.tile, g = it.g, seg = it.seg;
    const int64_t b = it.b;
    const int ch0 = tile * 16 * C;
    const int64_t d0 = (int64_t)g * p.per + ch0;
    const int nch = p.per - ch0 < 16 * C ? p.per - ch0 : 16 * C;
    const int nv = nch - cl * C < 0 ? 0 : nch - cl * C > C ? C : nch - cl * C;
    const int64_t len = seq_len(p.lengths, b, p.T);
    const bool whole = C == 1 || p.vec;
    float A2[S][C], skip[C], bias[C], dA[S][C], dskip[C], dbias[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t d = d0 + cl * C + c;
        const bool ok = c < nv;
        skip[c] = ok && p.skip ? p.skip[d] : 0.f;
        bias[c] = ok && p.delta_bias ? p.delta_bias[d] : 0.f;
        dskip[c] = dbias[c] = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int n = sg * S + s;
            A2[s][c] = ok && n < p.N ? gate_base(p.A[d * p.N + n]) : 0.f;
            dA[s][c] = 0.f;
        }
    }
    // Folds: thread tid takes tasks tid, tid + NT, ...; task i < E folds the states
    // of position i forward, task E + i the gradients in reverse.  `edge` is what
    // enters the block: the saved state before it, the gradient from its right.
    float edge[FPT];
    int st_off[FPT];  // offset from the tile's first state, or -1
    const int64_t st_base = b * p.D * p.N + d0 * p.N;
#pragma unroll
    for (int f = 0; f < FPT; ++f) {
        const int i = tid + f * NT;
        int ln, e;
        LV::where(i % E, &ln, &e);
        const int n = (ln >> 4) * S + e % S, ch = (ln & 15) * C + e / S;
        st_off[f] = i < 2 * E && n < p.N && ch < nch ? ch * (int)p.N + n : -1;
        edge[f] = i >= E && st_off[f] >= 0 && p.dhT ? p.dhT[st_base + st_off[f]] : 0.f;
        if (i >= E && st_off[f] >= 0) {
            const float *v = p.seg_v + st_base + st_off[f], *q = p.seg_p + st_base + st_off[f];
#pragma unroll 4
            for (int k = p.n_seg - 1; k > seg; --k)
                edge[f] = carry_through(q[k * p.B * p.D * p.N], edge[f], v[k * p.B * p.D * p.N]);
        }
    }
    const uint32_t row = (uint32_t)(p.D * (int64_t)sizeof(T));
    uint32_t voff[J], boff[BPL];
#pragma unroll
    for (int j = 0; j < J; ++j)
        voff[j] = nv > 0 ? (uint32_t)(4 * j + sg) * row + (uint32_t)(cl * C * sizeof(T)) : NO_CHANNEL;
    const int64_t row0 = b * p.T * p.D + d0;
    const int64_t brow = (int64_t)p.G * p.N, b0 = (b * p.T * p.G + g) * p.N;
#pragma unroll
    for (int i = 0; i < BPL; ++i) {
        const int q = lane + 64 * i, t = q / NP, n = q % NP;
        boff[i] = q < L * NP && n < p.N ? (uint32_t)((t * brow + n) * (int64_t)sizeof(T)) : NO_CHANNEL;
    }
    const int64_t bc = p.B * p.T * brow;  // floats of dBm
    float *part_b = p.part_bc + (int64_t)tile * 2 * bc + b0;
    float *part_c = part_b + bc;
    const int64_t n_blk = (p.T + NW * L - 1) / (NW * L);
    raw_t ur[J], dr[J], zr[J], gr[J];
    one_t br[BPL], cr[BPL];

    // this wave's rows of a block, and the state before it
    const auto load = [&](int64_t blk) {
        const int64_t t0 = blk * (NW * L) + wave * L, left = steps_left<L>(t0, len);
        load_rows<T, C, J>(make_rows(static_cast<const T *>(p.u) + row0 + t0 * p.D, left * row), voff, nv, whole, ur);
        load_rows<T, C, J>(make_rows(static_cast<const T *>(p.delta) + row0 + t0 * p.D, left * row), voff, nv, whole,
                           dr);
        load_rows<T, C, J>(make_rows(static_cast<const T *>(p.dy) + row0 + t0 * p.D, left * row), voff, nv, whole, gr);
        if constexpr (GATED)
            load_rows<T, C, J>(make_rows(static_cast<const T *>(p.z) + row0 + t0 * p.D, left * row), voff, nv, whole,
                               zr);
        const rsrc_t rb = make_rows(static_cast<const T *>(p.Bm) + b0 + t0 * brow, left * brow * (int64_t)sizeof(T));
        const rsrc_t rc = make_rows(static_cast<const T *>(p.Cm) + b0 + t0 * brow, left * brow * (int64_t)sizeof(T));
#pragma unroll
        for (int i = 0; i < BPL; ++i) {
            br[i] = buf_read<T, 1>(rb, boff[i]);
            cr[i] = buf_read<T, 1>(rc, boff[i]);
        }
        const float *st = p.states + (b * n_blk + blk) * p.D * p.N + d0 * p.N;
#pragma unroll
        for (int f = 0; f < FPT; ++f)
            if (tid + f * NT < E) edge[f] = st_off[f] >= 0 ? st[st_off[f]] : 0.f;
    };

    const int64_t blk0 = seg * (p.seg / (NW * L)), end = blk0 + p.seg / (NW * L);
    // blocks past the sequence's end pass the gradient on and have zero rows
    const int64_t last = end < n_blk ? end : n_blk, live = (len + NW * L - 1) / (NW * L);
    const int64_t blk1 = last < live ? last : live > blk0 ? live : blk0;
    for (int64_t blk = blk1; blk < last; ++blk) {
        const int64_t t0 = blk * (NW * L) + wave * L;
        const int rows = steps_left<L>(t0, p.T);
        const float zero[C] = {};
        const int64_t at = row0 + t0 * p.D;
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (4 * j + sg < rows) {
                store_ch<T, C>(reinterpret_cast<char *>(static_cast<T *>(p.du) + at) + voff[j], nv, whole, zero);
                store_ch<T, C>(reinterpret_cast<char *>(static_cast<T *>(p.ddelta) + at) + voff[j], nv, whole, zero);
                if constexpr (GATED)
                    store_ch<T, C>(reinterpret_cast<char *>(static_cast<T *>(p.dz) + at) + voff[j], nv, whole, zero);
            }
        for (int q = lane; q < L * NP; q += 64)
            if (q / NP < rows && q % NP < p.N) {
                part_b[(t0 + q / NP) * brow + q % NP] = 0.f;
                part_c[(t0 + q / NP) * brow + q % NP] = 0.f;
            }
    }
    if (blk1 > blk0) load(blk1 - 1);
    for (int64_t blk = blk1 - 1; blk >= blk0; --blk) {
        const int64_t t0 = blk * (NW * L) + wave * L;
        const int left = steps_left<L>(t0, len), rows = steps_left<L>(t0, p.T);
        {
            float uu[J * C], der[J * C], gz[J * C];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float u[C], dd[C], z[C], gy[C], x[2 * C];
                PC::unpack(ur[j], u);
                PC::unpack(dr[j], dd);
                PC::unpack(gr[j], gy);
                if constexpr (GATED) PC::unpack(zr[j], z);
                const bool in = 4 * j + sg < left;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float r = gate_rate(dd[c] + bias[c], p.softplus, &der[j * C + c]);
                    x[c] = in ? r : 0.f;
                    x[C + c] = x[c] * u[c];
                    uu[j * C + c] = u[c];
                    if constexpr (GATED) {
                        const float sig = sigmoid(z[c]);
                        gz[j * C + c] = gy[c] * dsilu(z[c], sig);
                        gy[c] *= z[c] * sig;
                    }
                }
                lds_write<2 * C>(my.x[4 * j + sg][cl], x);
                lds_write<C>(my.ds[4 * j + sg][cl], gy);
            }
            lds_write<J * C>(my.keep[0][lane], uu);
            lds_write<J * C>(my.keep[1][lane], der);
            if constexpr (GATED) lds_write<J * C>(my.keep[2][lane], gz);
        }
#pragma unroll
        for (int i = 0; i < BPL; ++i) {
            const int q = lane + 64 * i, t = q / NP, n = q % NP;
            if (L * NP % 64 == 0 || q < L * NP) {
                Pack<T, 1>::unpack(br[i], &my.b[t][n]);
                Pack<T, 1>::unpack(cr[i], &my.c[t][n]);
            }
        }
        wave_lds_sync();
        // local scans, forward and reverse
        float a[L][S][C];
        float hv[EL], gv[EL];
        {
            float sum[C];
#pragma unroll
            for (int c = 0; c < C; ++c) sum[c] = 0.f;
#pragma unroll
            for (int t = 0; t < L; ++t) {
                __builtin_amdgcn_sched_barrier(0);
                float x[2 * C], bt[S];
                lds_read<2 * C>(my.x[t][cl], x);
                lds_read<S>(&my.b[t][sg * S], bt);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    sum[c] += x[c];
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        a[t][s][c] = __builtin_amdgcn_exp2f(x[c] * A2[s][c]);
                        const float xb = bt[s] * x[C + c];
                        hv[c * S + s] = t == 0 ? xb : fmaf(a[t][s][c], hv[c * S + s], xb);
                    }
                }
                pin(hv);
            }
            LV::write(my.s, lane, hv);
#pragma unroll
            for (int t = L - 1; t >= 0; --t) {
                __builtin_amdgcn_sched_barrier(0);
                float gs[C], ct[S];
                lds_read<C>(my.ds[t][cl], gs);
                lds_read<S>(&my.c[t][sg * S], ct);
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        gv[c * S + s] =
                            a[t][s][c] * (t == L - 1 ? ct[s] * gs[c] : fmaf(ct[s], gs[c], gv[c * S + s]));
                pin(gv);
            }
            LV::write(my.r, lane, gv);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int s = 0; s < S; ++s) hv[c * S + s] = root_product(sum[c] * A2[s][c]);
            LV::write(my.p, lane, hv);
        }
        wg_lds_sync();
#pragma unroll
        for (int f = 0; f < FPT; ++f) {
            const int task = tid + f * NT;
            if (task < 2 * E) {
                // forward: s and p of waves 0, 1, ...; reverse: r and p of waves NW - 1, ...
                const bool rev = task >= E;
                const int i = rev ? task - E : task;
                WaveColumn<W, NW> val(smem, (int)(rev ? offsetof(W, r) : offsetof(W, s)) + i * 4);
                const WaveColumn<W, NW> gate(smem, (int)offsetof(W, p) + i * 4);
                float c = edge[f], pw[NW], v[NW];
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    pw[w] = gate[w];
                    v[w] = val[w];
                }
                if (rev) {
#pragma unroll
                    for (int w = NW - 1; w >= 0; --w) {
                        val[w] = c;
                        c = carry_through(pw[w], c, v[w]);
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        val[w] = c;
                        c = carry_through(pw[w], c, v[w]);
                    }
                }
                if (rev) edge[f] = c;
            }
        }
        wg_lds_sync();
        LV::read(my.s, lane, hv);
        wave_lds_sync();
        // states: keep a_t h_{t-1}; s_t for the gate's gradient; dCm
        float sv[4][C], ah[KEEP ? L : 1][S][C];
#pragma unroll
        for (int tq = 0; tq < L; tq += 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = tq + k;
                __builtin_amdgcn_sched_barrier(0);
                float x[2 * C], gs[C], bt[S], ct[S], dc[S];
                lds_read<2 * C>(my.x[t][cl], x);
                lds_read<C>(my.ds[t][cl], gs);
                lds_read<S>(&my.b[t][sg * S], bt);
                if constexpr (GATED) lds_read<S>(&my.c[t][sg * S], ct);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    sv[k][c] = 0.f;
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        float &h = hv[c * S + s];
                        const float p_h = a[t][s][c] * h;
                        if constexpr (KEEP) ah[t][s][c] = p_h;
                        else a[t][s][c] = p_h;
                        h = fmaf(bt[s], x[C + c], p_h);
                        if constexpr (GATED) sv[k][c] = fmaf(ct[s], h, sv[k][c]);
                        dc[s] = c == 0 ? gs[c] * h : fmaf(gs[c], h, dc[s]);
                    }
                }
                pin(hv);
                if constexpr (GATED) pin(sv[k]);
                lds_write<S>(&my.join[cl][sg * V + t % TR * S], dc);
                if (t % TR == TR - 1) {
                    wave_lds_sync();
                    join_channels<S, TR>(my.join, lane, [&](int tr, int n, float v) {
                        const int tl = t - (TR - 1) + tr;
                        if (tl < rows && n < p.N) part_c[(t0 + tl) * brow + n] = v;
                    });
                    wave_lds_sync();
                }
            }
            if constexpr (GATED) {  // four steps' s are complete: dz
                float so[C], uu[C], gz[C], o[C];
                sg_join4(sv[0], sv[1], sv[2], sv[3], so);
                lds_read<C>(&my.keep[0][lane][tq / 4 * C], uu);
                lds_read<C>(&my.keep[2][lane][tq / 4 * C], gz);
#pragma unroll
                for (int c = 0; c < C; ++c) o[c] = tq + sg < left ? gz[c] * fmaf(skip[c], uu[c], so[c]) : 0.f;
                if (tq + sg < rows)
                    store_ch<T, C>(reinterpret_cast<char *>(static_cast<T *>(p.dz) + row0 + t0 * p.D) + voff[tq / 4],
                                   nv, whole, o);
            }
        }
        // g in reverse and everything that depends on it
        LV::read(my.r, lane, gv);
        float dxv[4][C], dd2[4][C];
        for_each<L>([&](auto ri) {
            constexpr int t = L - 1 - decltype(ri)::value;
            __builtin_amdgcn_sched_barrier(0);
            float x[2 * C], gs[C], bt[S], ct[S], db[S];
            lds_read<2 * C>(my.x[t][cl], x);
            lds_read<C>(my.ds[t][cl], gs);
            lds_read<S>(&my.b[t][sg * S], bt);
            lds_read<S>(&my.c[t][sg * S], ct);
            float (&dx)[C] = dxv[t % 4], (&dd)[C] = dd2[t % 4];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                dx[c] = dd[c] = 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const float gt = fmaf(ct[s], gs[c], gv[c * S + s]);
                    float q;
                    if constexpr (KEEP) {
                        gv[c * S + s] = a[t][s][c] * gt;
                        q = gt * ah[t][s][c];
                    } else {
                        gv[c * S + s] = t > 0 ? __builtin_amdgcn_exp2f(x[c] * A2[s][c]) * gt : 0.f;
                        q = gt * a[t][s][c];
                    }
                    dx[c] = fmaf(gt, bt[s], dx[c]);
                    db[s] = c == 0 ? gt * x[C + c] : fmaf(gt, x[C + c], db[s]);
                    dd[c] = fmaf(q, A2[s][c], dd[c]);
                    dA[s][c] = fmaf(q, x[c], dA[s][c]);
                }
            }
            pin(dx);
            pin(dd);
#pragma unroll
            for (int s = 0; s < S; ++s) pin(dA[s]);
            lds_write<S>(&my.join[cl][sg * V + t % TR * S], db);
            if constexpr (t % TR == 0) {
                wave_lds_sync();
                join_channels<S, TR>(my.join, lane, [&](int tr, int n, float v) {
                    const int tl = t + tr;
                    if (tl < rows && n < p.N) part_b[(t0 + tl) * brow + n] = v;
                });
                wave_lds_sync();
            }
            if constexpr (t == L / 2) {  // half the gates are done with: registers for the next block's rows
                if (blk > blk0) load(blk - 1);
            }
            if constexpr (t % 4 == 0) {  // four steps are complete: their rows
                constexpr int j = t / 4;
                float xo[C], ao[C], o1[C], o2[C], uu[C], der[C], xr[2 * C], dsr[C];
                sg_join4(dxv[0], dxv[1], dxv[2], dxv[3], xo);
                sg_join4(dd2[0], dd2[1], dd2[2], dd2[3], ao);
                lds_read<C>(&my.keep[0][lane][j * C], uu);
                lds_read<C>(&my.keep[1][lane][j * C], der);
                lds_read<2 * C>(my.x[t + sg][cl], xr);
                lds_read<C>(my.ds[t + sg][cl], dsr);
                const bool in = t + sg < left;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    o1[c] = in ? fmaf(xr[c], xo[c], skip[c] * dsr[c]) : 0.f;
                    o2[c] = in ? fmaf(uu[c], xo[c], LN2 * ao[c]) * der[c] : 0.f;
                    dskip[c] = fmaf(dsr[c], uu[c], dskip[c]);
                    dbias[c] += o2[c];
                }
                if (t + sg < rows) {
                    const int64_t at = row0 + t0 * p.D;
                    store_ch<T, C>(reinterpret_cast<char *>(static_cast<T *>(p.du) + at) + voff[j], nv, whole, o1);
                    store_ch<T, C>(reinterpret_cast<char *>(static_cast<T *>(p.ddelta) + at) + voff[j], nv, whole, o2);
                }
            }
        });
    }
#pragma unroll
    for (int f = 0; f < FPT; ++f)
        if (tid + f * NT >= E && st_off[f] >= 0 && p.dh0 && seg == 0) p.dh0[st_base + st_off[f]] = edge[f];
    // dA over the waves; dskip and ddelta_bias over the waves and lane rows too
    float ev[EL], kb[2 * C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        kb[c] = dskip[c];
        kb[C + c] = dbias[c];
#pragma unroll
        for (int s = 0; s < S; ++s) ev[c * S + s] = dA[s][c];
    }
    LV::write(my.r, lane, ev);
    lds_write<2 * C>(my.x[sg][cl], kb);
    wg_lds_sync();
    float *pa = p.part_a + (b * p.n_seg + seg) * (p.N + 2) * p.D;
#pragma unroll
    for (int f = 0; f < FPT; ++f) {
        const int i = tid + f * NT;
        if (i < E && st_off[f] >= 0) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) s += sm[w].r[i];
            const int ch = st_off[f] / (int)p.N, n = st_off[f] - ch * (int)p.N;
            pa[n * p.D + d0 + ch] = s;
        }
    }
    if (tid < 16 * 2 * C) {
        const int l = tid / (2 * C), k = tid % (2 * C), c = k % C;
        if (l * C + c < nch) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w)
#pragma unroll
                for (int q = 0; q < 4; ++q) s += sm[w].x[q][l][k];
            pa[(p.N + k / C) * p.D + d0 + l * C + c] = s;
        }
    }
}

template <typename T>
struct StoreShared {
    T *dB, *dC;
    int64_t half;
    __device__ __forceinline__ void operator()(int64_t m, float s) const {
        if (m < half) st1(dB + m, s);
        else st1(dC + m - half, s);
    }
};

struct StoreParams {
    float *dA, *dskip, *dbias;
    int64_t D, N;
    __device__ __forceinline__ void operator()(int64_t m, float s) const {
        const int64_t k = m / D, d = m - k * D;
        if (k < N) dA[d * N + k] = s;
        else if (k == N) {
            if (dskip) dskip[d] = s;
        } else if (dbias) {
            dbias[d] = s;
        }
    }
};

int64_t bwd_tiles(int64_t per, int64_t N) {
    const int S = scan_s(N);
    const int64_t w = 16 * (S <= 4 ? 2 : 1);
    return (per + w - 1) / w;
}

// Segments of the backward: as many as make at most 256 workgroups, since the LDS holds
// one a CU: more would run in a second turn.  B = 1, T = 4096, N = 16, bf16: 40 tiles 133
// us in 6 segments and 205 in 7, 90 tiles 335 in 2 and 408 in 3; 160 tiles 507 uncut and
// 588 in 2; N = 4 and 64 alike (90 tiles: 189 and 232, 807 and 957).
int64_t bwd_segments(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    const int64_t n = B * G * bwd_tiles(D / G, N), blk = scan_block(N), blocks = (T + blk - 1) / blk;
    if (n > 128 || blocks < 3) return 1;  // (a launch costs the host about half a block's time)
    const int64_t want = 256 / n, seg = (blocks + want - 1) / want;
    return (blocks + seg - 1) / seg;
}

template <typename T, int S>
mi_status launch_bwd(ScanArgs a, hipStream_t s) {
    using TL = BwdTile<S>;
    constexpr int SH = TL::NW * (int)sizeof(BwdWave<S, TL::C, TL::L>);
    static_assert(SH <= 160 * 1024, "a workgroup's LDS");
    constexpr int64_t BLK = TL::NW * TL::L;
    a.tiles = (int)bwd_tiles(a.per, a.N);
    a.seg = (a.T + BLK * a.n_seg - 1) / (BLK * a.n_seg) * BLK;
    int64_t items;
    if (!mul_ok(a.B, a.G, a.tiles, a.n_seg, &items) || !launch_fits(items + 7, TL::NW * 64)) return MI_ERR_UNSUPPORTED;
    if (a.n_seg > 1) {
        a.n_items = (int)(items / a.n_seg * (a.n_seg - 1));
        hipLaunchKernelGGL((scan_bwd_sum_kernel<T, S, TL::C, TL::L, TL::NW>), dim3(xcd_grid(a.n_items)),
                           dim3(TL::NW * 64), 0, s, a);
        const mi_status st = launch_status();
        if (st != MI_OK) return st;
    }
    a.n_items = (int)items;
    const auto kernel = a.z ? scan_bwd_kernel<T, S, TL::C, TL::L, TL::NW, true>
                            : scan_bwd_kernel<T, S, TL::C, TL::L, TL::NW, false>;
    if (hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                            SH) != hipSuccess)
        return MI_ERR_LAUNCH;
    hipLaunchKernelGGL(kernel, dim3(xcd_grid(a.n_items)), dim3(TL::NW * 64), SH, s, a);
    return launch_status();
}
template <typename T>
mi_status launch_bwd_t(const ScanArgs &a, void *dBm, void *dCm, const StoreParams &params, hipStream_t s) {
    mi_status st = MI_OK;
    if (a.B > 0) switch (scan_s(a.N)) {
            case 1: st = launch_bwd<T, 1>(a, s); break;
            case 2: st = launch_bwd<T, 2>(a, s); break;
            case 4: st = launch_bwd<T, 4>(a, s); break;
            case 8: st = launch_bwd<T, 8>(a, s); break;
            default: st = launch_bwd<T, 16>(a, s);
        }
    if (st != MI_OK) return st;
    const int64_t bc = a.B * a.T * a.G * a.N;
    const auto shared = reduce_of(a.part_bc, bwd_tiles(a.per, a.N), 2 * bc,
                                  StoreShared<T>{static_cast<T *>(dBm), static_cast<T *>(dCm), bc});
    const auto own = reduce_of(a.part_a, a.B * a.n_seg, (a.N + 2) * a.D, params);
    hipLaunchKernelGGL((reduce_two_kernel<StoreShared<T>, StoreParams>), dim3((unsigned)(shared.blocks + own.blocks)),
                       dim3(256), 0, s, shared, own);
    return launch_status();
}

// Workspace: partial dBm and dCm; partial dA, dskip, ddelta_bias; the segments'
// transforms.
struct BwdWs {
    int64_t bc, a, n_seg, total;  // bytes, bytes, segments, bytes
};
bool bwd_ws(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, BwdWs *w) {
    int64_t x, y, v;
    w->n_seg = bwd_segments(B, T, D, G, N);
    if (!mul_ok(B, T, G, N, &x) || !mul_ok(x, bwd_tiles(D / G, N), 8, 1, &x) ||
        !mul_ok(B * w->n_seg, N + 2, D, 4, &y) || !mul_ok(w->n_seg > 1 ? B * w->n_seg : 0, N, D, 8, &v))
        return false;
    w->bc = (int64_t)round_up((size_t)x, 256);
    w->a = (int64_t)round_up((size_t)y, 256);
    return !__builtin_add_overflow(w->bc, w->a, &w->total) && !__builtin_add_overflow(w->total, v, &w->total);
}

}  // namespace
}  // namespace miscan

using namespace miscan;

extern "C" {

size_t mi_selective_scan_bwd_workspace(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, mi_dtype dt) {
    ScanSizes s;
    BwdWs w;
    if (check_scan(B, T, D, G, N, dt, &s) != MI_OK || B == 0 || D == 0 || !bwd_ws(B, T, D, G, N, &w)) return 0;
    return (size_t)w.total;
}

mi_status mi_selective_scan_bwd(const void *u, const void *delta, const float *A, const void *Bm, const void *Cm,
                                const float *skip, const void *z, const float *delta_bias, const float *states,
                                const int32_t *lengths, const void *dy, const float *dhT, void *du, void *ddelta,
                                float *dA, void *dBm, void *dCm, float *dskip, void *dz, float *ddelta_bias,
                                float *dh0, int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, int softplus_on,
                                mi_dtype dt, void *ws, size_t ws_bytes, hipStream_t stream) {
    ScanSizes s;
    mi_status st = check_scan(B, T, D, G, N, dt, &s);
    if (st != MI_OK) return st;
    // gradients go with their inputs
    if ((skip == nullptr) != (dskip == nullptr) || (z == nullptr) != (dz == nullptr) ||
        (delta_bias == nullptr) != (ddelta_bias == nullptr))
        return MI_ERR_INVALID_ARG;
    if (D == 0) return MI_OK;
    const size_t es = elem_size(dt);
    BufList in, out;
    in.need(u, s.x, es).need(delta, s.x, es).need(A, s.a, 4).need(Bm, s.bc, es).need(Cm, s.bc, es);
    in.opt(skip, s.d, 4).opt(z, s.x, es).opt(delta_bias, s.d, 4).need(states, s.states, 4);
    in.opt(lengths, B * 4, 4).need(dy, s.x, es).opt(dhT, s.h, 4);
    out.need(du, s.x, es).need(ddelta, s.x, es).need(dA, s.a, 4).need(dBm, s.bc, es).need(dCm, s.bc, es);
    out.opt(dskip, s.d, 4).opt(dz, s.x, es).opt(ddelta_bias, s.d, 4).opt(dh0, s.h, 4);
    if ((st = check_lists(in, out)) != MI_OK) return st;
    ScanArgs a{};
    a.u = u; a.delta = delta; a.z = z; a.Bm = Bm; a.Cm = Cm; a.A = A; a.skip = skip; a.delta_bias = delta_bias;
    a.lengths = lengths; a.states = const_cast<float *>(states); a.dy = dy; a.dhT = dhT; a.du = du;
    a.ddelta = ddelta; a.dz = dz; a.dh0 = dh0;
    a.B = B; a.T = T; a.D = D; a.N = N; a.softplus = softplus_on != 0;
    if (D > SCAN_MAX_D || G * N > SCAN_MAX_D) return MI_ERR_UNSUPPORTED;
    a.G = (int)G; a.per = (int)(D / G);
    a.vec = scan_vec(a, dt);
    if (B > 0) {
        BwdWs w;
        if (!bwd_ws(B, T, D, G, N, &w)) return MI_ERR_INVALID_ARG;
        if ((st = check_ws_lists(ws, ws_bytes, (size_t)w.total, in, out)) != MI_OK) return st;
        a.part_bc = static_cast<float *>(ws);
        a.part_a = reinterpret_cast<float *>(static_cast<char *>(ws) + w.bc);
        a.n_seg = (int)w.n_seg;
        a.seg_v = reinterpret_cast<float *>(static_cast<char *>(ws) + w.bc + w.a);
        a.seg_p = a.seg_v + w.n_seg * B * D * N;
    }
    const StoreParams params{dA, dskip, ddelta_bias, D, N};
    if (dt == MI_F32) return launch_bwd_t<float>(a, dBm, dCm, params, stream);
    if (dt == MI_BF16) return launch_bwd_t<bf16_t>(a, dBm, dCm, params, stream);
    return launch_bwd_t<f16_t>(a, dBm, dCm, params, stream);
}

}  // extern "C"
