// selective_scan_bwd.hip -- gradient of the selective state-space scan.
//
// A workgroup walks the blocks of one channel tile in reverse, each from the
// state the forward saved before it.  Inside a block every wave scans its steps
// forward (states) and in reverse (g a) from zero, one meeting in LDS folds both
// carries, and every wave then runs its steps forward from its true state
// (keeping a_t h_{t-1}) and in reverse from its true g.  Per state-step: gate 3
// issue slots (mul, exp2), local scans 4, states 2 to 4, gradients 7.
//
// dBm and dCm sum over the channels of a group: C of them in the lane, sixteen
// lanes through LDS, the tiles of a group through partial rows that
// reduce_parts adds in a fixed order.
#include "checks.hpp"
#include "selective_scan.hpp"

namespace miscan {
namespace {

// Steps joined over the channel lanes at once: 32 values a lane, 16 for S = 16
// (LDS).
constexpr int join_steps(int S, int L) { return S == 16 ? 1 : 32 / S < L ? 32 / S : L; }

template <int S, int C, int L, int NW>
struct BwdShared {
    static constexpr int E = S * C * 64, TR = join_steps(S, L), V = TR * S, ROW = 4 * V + 4;
    float x[NW][L][16][2 * C];   // dl, dl u
    float ds[NW][L][16][C];
    static constexpr bool BY_STATE = S < 16;  // room for both orders of Bm
    float bt[NW][BY_STATE ? 4 * S : 1][L + 4];  // Bm by state
    float b[NW][L][4 * S];       // Bm by step
    float c[NW][L][4 * S];       // Cm by step
    float s[NW][E], p[NW][E], r[NW][E];
    float red[NW][16][ROW];      // values to sum over the channel lanes; rows four banks apart
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

template <typename T, int S, int C, int L, int NW, bool GATED>
__global__ __launch_bounds__(NW * 64, 2) void scan_bwd_kernel(ScanArgs p) {
    constexpr int EL = S * C, J = L / 4, NP = 4 * S;
    constexpr int E = EL * 64, NT = NW * 64, FPT = (E + NT - 1) / NT, BPL = (L * NP + 63) / 64;
    using LV = LaneVec<EL>;
    using QR = QuadRow<S>;
    constexpr int NB = QR::NB;
    using PC = Pack<T, C>;
    using raw_t = typename PC::raw_t;
    using one_t = typename Pack<T, 1>::raw_t;
    using SH = BwdShared<S, C, L, NW>;
    constexpr int TR = SH::TR, V = SH::V;
    constexpr bool BY_STATE = SH::BY_STATE;
    extern __shared__ __align__(16) char smem[];
    SH &sm = *reinterpret_cast<SH *>(smem);
    const int item = xcd_item(p.n_items);
    if (item >= p.n_items) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int sg = lane >> 4, cl = lane & 15;
    const int tile = item % p.tiles;
    const int g = item / p.tiles % p.G;
    const int64_t b = item / p.tiles / p.G;
    const int ch0 = tile * 16 * C;
    const int64_t d0 = (int64_t)g * p.per + ch0;
    const int nch = p.per - ch0 < 16 * C ? p.per - ch0 : 16 * C;
    const int nv = nch - cl * C < 0 ? 0 : nch - cl * C > C ? C : nch - cl * C;
    const int64_t len = seq_len(p.lengths, b, p.T);
    const bool whole = p.vec && nch == 16 * C;
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
            A2[s][c] = ok && n < p.N ? p.A[d * p.N + n] * LOG2E : 0.f;
            dA[s][c] = 0.f;
        }
    }
    float carry[FPT], h0[FPT];  // gradient that enters the block from its right; state before the block
    int st_off[FPT];            // offset from the tile's first state, or -1
    const int64_t st_base = b * p.D * p.N + d0 * p.N;
#pragma unroll
    for (int f = 0; f < FPT; ++f) {
        const int i = tid + f * NT;
        int ln, e;
        LV::where(i < E ? i : 0, &ln, &e);
        const int n = (ln >> 4) * S + e % S, ch = (ln & 15) * C + e / S;
        st_off[f] = i < E && n < p.N && ch < nch ? ch * (int)p.N + n : -1;
        carry[f] = st_off[f] >= 0 && p.dhT ? p.dhT[st_base + st_off[f]] : 0.f;
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
    const int n0 = QR::first(lane);
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
        for (int f = 0; f < FPT; ++f) h0[f] = st_off[f] >= 0 ? st[st_off[f]] : 0.f;
    };

    if (n_blk > 0) load(n_blk - 1);
    for (int64_t blk = n_blk - 1; blk >= 0; --blk) {
        const int64_t t0 = blk * (NW * L) + wave * L;
        const int left = steps_left<L>(t0, len), rows = steps_left<L>(t0, p.T);
        raw_t uk[J], zk[J], gk[J];
        float der[J][C], hin[FPT];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float uu[C], dd[C], zz[C], gy[C];
            PC::unpack(ur[j], uu);
            PC::unpack(dr[j], dd);
            PC::unpack(gr[j], gy);
            if constexpr (GATED) PC::unpack(zr[j], zz);
            uk[j] = ur[j];
            gk[j] = gr[j];
            if constexpr (GATED) zk[j] = zr[j];
            const bool in = 4 * j + sg < left;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float r = gate_rate(dd[c] + bias[c], p.softplus, &der[j][c]);
                r = in ? r : 0.f;
                sm.x[wave][4 * j + sg][cl][c] = r;
                sm.x[wave][4 * j + sg][cl][C + c] = r * uu[c];
                if constexpr (GATED) gy[c] *= silu(zz[c]);
                sm.ds[wave][4 * j + sg][cl][c] = gy[c];
            }
        }
#pragma unroll
        for (int i = 0; i < BPL; ++i) {
            const int q = lane + 64 * i, t = q / NP, n = q % NP;
            if (L * NP % 64 == 0 || q < L * NP) {
                float f;
                Pack<T, 1>::unpack(br[i], &f);
                if constexpr (BY_STATE) sm.bt[wave][n][t] = f;
                sm.b[wave][t][n] = f;
                Pack<T, 1>::unpack(cr[i], &sm.c[wave][t][n]);
            }
        }
#pragma unroll
        for (int f = 0; f < FPT; ++f) hin[f] = h0[f];
        if (blk > 0) load(blk - 1);
        wave_lds_sync();
        // local scans, forward and reverse
        float a[L][S][C];
        float hv[EL], gv[EL];
        {
            float sum[C];
#pragma unroll
            for (int c = 0; c < C; ++c) sum[c] = 0.f;
#pragma unroll
            for (int tq = 0; tq < L; tq += 4) {
                float bq[NB][4];
#pragma unroll
                for (int i = 0; i < NB; ++i)
                    if constexpr (BY_STATE) lds_read<4>(&sm.bt[wave][n0 + 4 * i][tq], bq[i]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int t = tq + k;
                    __builtin_amdgcn_sched_barrier(0);
                    float x[2 * C], bt[NB], bw[S];
                    lds_read<2 * C>(sm.x[wave][t][cl], x);
#pragma unroll
                    for (int i = 0; i < NB; ++i)
                        if constexpr (BY_STATE) bt[i] = bq[i][k];
                    if constexpr (!BY_STATE) lds_read<S>(&sm.b[wave][t][sg * S], bw);
#pragma unroll
                    for (int c = 0; c < C; ++c) sum[c] += x[c];
                    for_each<S>([&](auto si) {
                        constexpr int s = decltype(si)::value;
                        float bs;
                        if constexpr (BY_STATE) bs = QR::template get<s>(bt);
                        else bs = bw[s];
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            a[t][s][c] = __builtin_amdgcn_exp2f(x[c] * A2[s][c]);
                            const float xb = bs * x[C + c];
                            hv[c * S + s] = t == 0 ? xb : fmaf(a[t][s][c], hv[c * S + s], xb);
                        }
                    });
                    pin(hv);
                }
            }
            LV::write(sm.s[wave], lane, hv);
#pragma unroll
            for (int t = L - 1; t >= 0; --t) {
                __builtin_amdgcn_sched_barrier(0);
                float gs[C], ct[S];
                lds_read<C>(sm.ds[wave][t][cl], gs);
                lds_read<S>(&sm.c[wave][t][sg * S], ct);
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        gv[c * S + s] =
                            a[t][s][c] * (t == L - 1 ? ct[s] * gs[c] : fmaf(ct[s], gs[c], gv[c * S + s]));
                pin(gv);
            }
            LV::write(sm.r[wave], lane, gv);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int s = 0; s < S; ++s) hv[c * S + s] = __builtin_amdgcn_exp2f(sum[c] * A2[s][c]);
            LV::write(sm.p[wave], lane, hv);
        }
        wg_lds_sync();
#pragma unroll
        for (int f = 0; f < FPT; ++f) {
            const int i = tid + f * NT;
            if (i < E) {
                float h = hin[f], gc = carry[f], pw[NW], sv[NW], rv[NW];
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    pw[w] = sm.p[w][i];
                    sv[w] = sm.s[w][i];
                    rv[w] = sm.r[w][i];
                }
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    sm.s[w][i] = h;
                    h = fmaf(pw[w], h, sv[w]);
                    sm.r[NW - 1 - w][i] = gc;
                    gc = fmaf(pw[NW - 1 - w], gc, rv[NW - 1 - w]);
                }
                carry[f] = gc;
            }
        }
        wg_lds_sync();
        LV::read(sm.s[wave], lane, hv);
        // states: keep a_t h_{t-1}; s_t for the gate's gradient; dCm
        float ah[L][S][C], sv[4][C], so[J][C];
#pragma unroll
        for (int tq = 0; tq < L; tq += 4) {
            float bq[NB][4];
#pragma unroll
            for (int i = 0; i < NB; ++i)
                if constexpr (BY_STATE) lds_read<4>(&sm.bt[wave][n0 + 4 * i][tq], bq[i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = tq + k;
                __builtin_amdgcn_sched_barrier(0);
                float x[2 * C], gs[C], ct[S], bt[NB], bw[S], dc[S];
                lds_read<2 * C>(sm.x[wave][t][cl], x);
                lds_read<C>(sm.ds[wave][t][cl], gs);
                if constexpr (GATED) lds_read<S>(&sm.c[wave][t][sg * S], ct);
#pragma unroll
                for (int i = 0; i < NB; ++i)
                    if constexpr (BY_STATE) bt[i] = bq[i][k];
                if constexpr (!BY_STATE) lds_read<S>(&sm.b[wave][t][sg * S], bw);
#pragma unroll
                for (int c = 0; c < C; ++c) sv[k][c] = 0.f;
                for_each<S>([&](auto si) {
                    constexpr int s = decltype(si)::value;
                    float bs;
                    if constexpr (BY_STATE) bs = QR::template get<s>(bt);
                    else bs = bw[s];
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        float &h = hv[c * S + s];
                        ah[t][s][c] = a[t][s][c] * h;
                        h = fmaf(a[t][s][c], h, bs * x[C + c]);
                        if constexpr (GATED) sv[k][c] = fmaf(ct[s], h, sv[k][c]);
                        dc[s] = c == 0 ? gs[c] * h : fmaf(gs[c], h, dc[s]);
                    }
                });
                if constexpr (GATED) pin(sv[k]);
#pragma unroll
                for (int s = 0; s < S; ++s) sm.red[wave][cl][sg * V + t % TR * S + s] = dc[s];
                if (t % TR == TR - 1) {
                    wave_lds_sync();
                    join_channels<S, TR>(sm.red[wave], lane, [&](int tr, int n, float v) {
                        const int tl = t - (TR - 1) + tr;
                        if (tl < rows && n < p.N) part_c[(t0 + tl) * brow + n] = v;
                    });
                    wave_lds_sync();
                }
            }
            if constexpr (GATED) sg_join4(sv[0], sv[1], sv[2], sv[3], so[tq / 4]);
        }
        // g in reverse and everything that depends on it
        LV::read(sm.r[wave], lane, gv);
        float dxv[4][C], dd2[4][C];
#pragma unroll
        for (int t = L - 1; t >= 0; --t) {
            __builtin_amdgcn_sched_barrier(0);
            float x[2 * C], gs[C], bt[S], ct[S], db[S];
            lds_read<2 * C>(sm.x[wave][t][cl], x);
            lds_read<C>(sm.ds[wave][t][cl], gs);
            lds_read<S>(&sm.b[wave][t][sg * S], bt);
            lds_read<S>(&sm.c[wave][t][sg * S], ct);
            float (&dx)[C] = dxv[t % 4], (&dd)[C] = dd2[t % 4];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                dx[c] = dd[c] = 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const float gt = fmaf(ct[s], gs[c], gv[c * S + s]);
                    gv[c * S + s] = a[t][s][c] * gt;
                    const float q = gt * ah[t][s][c];
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
#pragma unroll
            for (int s = 0; s < S; ++s) sm.red[wave][cl][sg * V + t % TR * S + s] = db[s];
            if (t % TR == 0) {
                wave_lds_sync();
                join_channels<S, TR>(sm.red[wave], lane, [&](int tr, int n, float v) {
                    const int tl = t + tr;
                    if (tl < rows && n < p.N) part_b[(t0 + tl) * brow + n] = v;
                });
                wave_lds_sync();
            }
            if (t % 4 == 0) {  // four steps are complete: their rows
                const int j = t / 4;
                float xo[C], ao[C], o1[C], o2[C], o3[C], uu[C], zz[C], gy[C], xr[2 * C], dsr[C];
                sg_join4(dxv[0], dxv[1], dxv[2], dxv[3], xo);
                sg_join4(dd2[0], dd2[1], dd2[2], dd2[3], ao);
                PC::unpack(uk[j], uu);
                PC::unpack(gk[j], gy);
                if constexpr (GATED) PC::unpack(zk[j], zz);
                lds_read<2 * C>(sm.x[wave][t + sg][cl], xr);
                lds_read<C>(sm.ds[wave][t + sg][cl], dsr);
                const bool in = t + sg < left;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    o1[c] = in ? fmaf(xr[c], xo[c], skip[c] * dsr[c]) : 0.f;
                    o2[c] = in ? fmaf(uu[c], xo[c], LN2 * ao[c]) * der[j][c] : 0.f;
                    dskip[c] = fmaf(dsr[c], uu[c], dskip[c]);
                    dbias[c] += o2[c];
                    if constexpr (GATED)
                        o3[c] = in ? gy[c] * fmaf(skip[c], uu[c], so[j][c]) * dsilu(zz[c], sigmoid(zz[c])) : 0.f;
                }
                if (t + sg < rows) {
                    const int64_t at = row0 + t0 * p.D;
                    store_ch<T, C>(reinterpret_cast<char *>(static_cast<T *>(p.du) + at) + voff[j], nv, whole, o1);
                    store_ch<T, C>(reinterpret_cast<char *>(static_cast<T *>(p.ddelta) + at) + voff[j], nv, whole, o2);
                    if constexpr (GATED)
                        store_ch<T, C>(reinterpret_cast<char *>(static_cast<T *>(p.dz) + at) + voff[j], nv, whole, o3);
                }
            }
        }
    }
#pragma unroll
    for (int f = 0; f < FPT; ++f)
        if (st_off[f] >= 0 && p.dh0) p.dh0[st_base + st_off[f]] = carry[f];
    // dA over the waves; dskip and ddelta_bias over the waves and lane rows too
    wg_lds_sync();
    float ev[EL];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int s = 0; s < S; ++s) ev[c * S + s] = dA[s][c];
    LV::write(sm.s[wave], lane, ev);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        sm.red[wave][cl][sg * 2 * C + c] = dskip[c];
        sm.red[wave][cl][sg * 2 * C + C + c] = dbias[c];
    }
    wg_lds_sync();
    float *pa = p.part_a + b * (p.N + 2) * p.D;
#pragma unroll
    for (int f = 0; f < FPT; ++f) {
        const int i = tid + f * NT;
        if (st_off[f] >= 0) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) s += sm.s[w][i];
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
                for (int q = 0; q < 4; ++q) s += sm.red[w][l][q * 2 * C + k];
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

template <typename T, int S>
mi_status launch_bwd(ScanArgs a, hipStream_t s) {
    using TL = ScanTile<S>;
    using SH = BwdShared<S, TL::C, TL::L, SCAN_NW>;
    static_assert(sizeof(SH) <= 160 * 1024, "a workgroup's LDS");
    a.tiles = (int)bwd_tiles(a.per, a.N);
    int64_t items;
    if (!mul_ok(a.B, a.G, a.tiles, 1, &items) || items > 0x7ffffff0) return MI_ERR_UNSUPPORTED;
    a.n_items = (int)items;
    const auto kernel = a.z ? scan_bwd_kernel<T, S, TL::C, TL::L, SCAN_NW, true>
                            : scan_bwd_kernel<T, S, TL::C, TL::L, SCAN_NW, false>;
    if (hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)sizeof(SH)) != hipSuccess)
        return MI_ERR_LAUNCH;
    hipLaunchKernelGGL(kernel, dim3(xcd_grid(a.n_items)), dim3(SCAN_NW * 64), sizeof(SH), s, a);
    return launch_status();
}
template <typename T>
mi_status launch_bwd_t(const ScanArgs &a, void *dBm, void *dCm, hipStream_t s) {
    mi_status st;
    switch (scan_s(a.N)) {
        case 1: st = launch_bwd<T, 1>(a, s); break;
        case 2: st = launch_bwd<T, 2>(a, s); break;
        case 4: st = launch_bwd<T, 4>(a, s); break;
        case 8: st = launch_bwd<T, 8>(a, s); break;
        default: st = launch_bwd<T, 16>(a, s);
    }
    if (st != MI_OK) return st;
    const int64_t bc = a.B * a.T * a.G * a.N;
    return reduce_parts(a.part_bc, bwd_tiles(a.per, a.N), 2 * bc,
                        StoreShared<T>{static_cast<T *>(dBm), static_cast<T *>(dCm), bc}, s);
}

// Workspace: partial dBm and dCm, then partial dA, dskip, ddelta_bias.
struct BwdWs {
    int64_t bc, total;
};
bool bwd_ws(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, BwdWs *w) {
    int64_t x, y;
    if (!mul_ok(B, T, G, N, &x) || !mul_ok(x, bwd_tiles(D / G, N), 8, 1, &x) || !mul_ok(B, N + 2, D, 4, &y)) return false;
    w->bc = (int64_t)round_up((size_t)x, 256);
    return !__builtin_add_overflow(w->bc, y, &w->total);
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
        if (dt == MI_F32) st = launch_bwd_t<float>(a, dBm, dCm, stream);
        else if (dt == MI_BF16) st = launch_bwd_t<bf16_t>(a, dBm, dCm, stream);
        else st = launch_bwd_t<f16_t>(a, dBm, dCm, stream);
        if (st != MI_OK) return st;
    }
    return reduce_parts(a.part_a, B, (N + 2) * D, StoreParams{dA, dskip, ddelta_bias, D, N}, stream);
}

}  // extern "C"
