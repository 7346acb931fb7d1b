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
    float b[NW][2][L][4 * S];    // Bm, Cm
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

template <typename T, int S, int C, int L, int NW>
__global__ __launch_bounds__(NW * 64) void scan_bwd_kernel(ScanArgs p) {
    constexpr int EL = S * C, J = L / 4, NP = 4 * S;
    constexpr int E = EL * 64, NT = NW * 64, FPT = (E + NT - 1) / NT, BPL = (L * NP + 63) / 64;
    using LV = LaneVec<EL>;
    using SH = BwdShared<S, C, L, NW>;
    constexpr int TR = SH::TR, V = SH::V;
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
    const int64_t dl0 = d0 + cl * C;
    const int64_t len = seq_len(p.lengths, b, p.T);
    const bool vec = p.vec;
    float A2[S][C], skip[C], bias[C], dA[S][C], dskip[C], dbias[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const bool ok = c < nv;
        skip[c] = ok && p.skip ? p.skip[dl0 + c] : 0.f;
        bias[c] = ok && p.delta_bias ? p.delta_bias[dl0 + c] : 0.f;
        dskip[c] = dbias[c] = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int n = sg * S + s;
            A2[s][c] = ok && n < p.N ? p.A[(dl0 + c) * p.N + n] * LOG2E : 0.f;
            dA[s][c] = 0.f;
        }
    }
    float carry[FPT];     // gradient that enters the block from its right
    int64_t st_off[FPT];  // offset in (D, N), or -1
#pragma unroll
    for (int f = 0; f < FPT; ++f) {
        const int i = tid + f * NT;
        int ln, e;
        LV::where(i < E ? i : 0, &ln, &e);
        const int n = (ln >> 4) * S + e % S, ch = (ln & 15) * C + e / S;
        st_off[f] = i < E && n < p.N && ch < nch ? (d0 + ch) * p.N + n : -1;
        carry[f] = st_off[f] >= 0 && p.dhT ? p.dhT[b * p.D * p.N + st_off[f]] : 0.f;
    }
    const int64_t row0 = b * p.T * p.D + dl0;
    const T *u = static_cast<const T *>(p.u) + row0;
    const T *delta = static_cast<const T *>(p.delta) + row0;
    const T *dy = static_cast<const T *>(p.dy) + row0;
    const T *z = p.z ? static_cast<const T *>(p.z) + row0 : nullptr;
    const T *Bm = static_cast<const T *>(p.Bm) + (b * p.T * p.G + g) * p.N;
    const T *Cm = static_cast<const T *>(p.Cm) + (b * p.T * p.G + g) * p.N;
    T *du = static_cast<T *>(p.du) + row0;
    T *ddelta = static_cast<T *>(p.ddelta) + row0;
    T *dz = p.z ? static_cast<T *>(p.dz) + row0 : nullptr;
    const int64_t brow = (int64_t)p.G * p.N;
    const int64_t bc = p.B * p.T * brow;  // floats of dBm
    float *part_b = p.part_bc + (int64_t)tile * 2 * bc + (b * p.T * p.G + g) * p.N;
    float *part_c = part_b + bc;
    const int64_t n_blk = (p.T + NW * L - 1) / (NW * L);

    for (int64_t blk = n_blk - 1; blk >= 0; --blk) {
        const int64_t t0 = blk * (NW * L) + wave * L;
        float h0[FPT];  // the state before the block
#pragma unroll
        for (int f = 0; f < FPT; ++f)
            h0[f] = st_off[f] >= 0 ? p.states[(b * n_blk + blk) * p.D * p.N + st_off[f]] : 0.f;
        float uu[J][C], zz[J][C], gy[J][C], dl[J][C], der[J][C], ds[J][C];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t t = t0 + 4 * j + sg;
            const int n_ok = t < len ? nv : 0;
            float dd[C];
            load_ch<T, C>(u + t * p.D, n_ok, vec, uu[j]);
            load_ch<T, C>(delta + t * p.D, n_ok, vec, dd);
            load_ch<T, C>(dy + t * p.D, n_ok, vec, gy[j]);
            if (z) load_ch<T, C>(z + t * p.D, n_ok, vec, zz[j]);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float r = gate_rate(dd[c] + bias[c], p.softplus, &der[j][c]);
                dl[j][c] = c < n_ok ? r : 0.f;
                ds[j][c] = z ? gy[j][c] * silu(zz[j][c]) : gy[j][c];
                sm.x[wave][4 * j + sg][cl][c] = dl[j][c];
                sm.x[wave][4 * j + sg][cl][C + c] = dl[j][c] * uu[j][c];
                sm.ds[wave][4 * j + sg][cl][c] = ds[j][c];
            }
        }
#pragma unroll
        for (int i = 0; i < BPL; ++i) {
            const int q = lane + 64 * i, t = q / NP, n = q % NP;
            const bool ok = q < L * NP && t0 + t < len && n < p.N;
            const float bv = ok ? ld1(Bm + (t0 + t) * brow + n) : 0.f;
            const float cv = ok ? ld1(Cm + (t0 + t) * brow + n) : 0.f;
            if (q < L * NP) {
                sm.b[wave][0][t][n] = bv;
                sm.b[wave][1][t][n] = cv;
            }
        }
        wave_lds_fence();
        // local scans, forward and reverse
        float a[L][S][C];
        float hv[EL], gv[EL];
        {
            float sum[C];
#pragma unroll
            for (int c = 0; c < C; ++c) sum[c] = 0.f;
#pragma unroll
            for (int e = 0; e < EL; ++e) hv[e] = gv[e] = 0.f;
#pragma unroll
            for (int t = 0; t < L; ++t) {
                float x[2 * C], bt[S];
                __builtin_amdgcn_sched_barrier(0);
                lds_read<2 * C>(sm.x[wave][t][cl], x);
                lds_read<S>(&sm.b[wave][0][t][sg * S], bt);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    sum[c] += x[c];
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        a[t][s][c] = __builtin_amdgcn_exp2f(x[c] * A2[s][c]);
                        hv[c * S + s] = fmaf(a[t][s][c], hv[c * S + s], x[C + c] * bt[s]);
                    }
                }
            }
#pragma unroll
            for (int t = L - 1; t >= 0; --t) {
                float gs[C], ct[S];
                __builtin_amdgcn_sched_barrier(0);
                lds_read<C>(sm.ds[wave][t][cl], gs);
                lds_read<S>(&sm.b[wave][1][t][sg * S], ct);
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        gv[c * S + s] = a[t][s][c] * fmaf(ct[s], gs[c], gv[c * S + s]);
            }
            LV::write(sm.s[wave], lane, hv);
            LV::write(sm.r[wave], lane, gv);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int s = 0; s < S; ++s) hv[c * S + s] = __builtin_amdgcn_exp2f(sum[c] * A2[s][c]);
            LV::write(sm.p[wave], lane, hv);
        }
        __syncthreads();
#pragma unroll
        for (int f = 0; f < FPT; ++f) {
            const int i = tid + f * NT;
            if (i < E) {
                float h = h0[f], gr = carry[f];
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float s = sm.s[w][i];
                    sm.s[w][i] = h;
                    h = fmaf(sm.p[w][i], h, s);
                }
#pragma unroll
                for (int w = NW - 1; w >= 0; --w) {
                    const float r = sm.r[w][i];
                    sm.r[w][i] = gr;
                    gr = fmaf(sm.p[w][i], gr, r);
                }
                carry[f] = gr;
            }
        }
        __syncthreads();
        LV::read(sm.s[wave], lane, hv);
        LV::read(sm.r[wave], lane, gv);
        // states: keep a_t h_{t-1}; s_t for the gate's gradient; dCm
        float ah[L][S][C], sv[L][C];
#pragma unroll
        for (int t = 0; t < L; ++t) {
            float x[2 * C], gs[C], bt[S], ct[S], dc[S];
            __builtin_amdgcn_sched_barrier(0);
            lds_read<2 * C>(sm.x[wave][t][cl], x);
            lds_read<C>(sm.ds[wave][t][cl], gs);
            lds_read<S>(&sm.b[wave][0][t][sg * S], bt);
            lds_read<S>(&sm.b[wave][1][t][sg * S], ct);
#pragma unroll
            for (int s = 0; s < S; ++s) dc[s] = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                sv[t][c] = 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    ah[t][s][c] = a[t][s][c] * hv[c * S + s];
                    hv[c * S + s] = fmaf(x[C + c], bt[s], ah[t][s][c]);
                    sv[t][c] = fmaf(ct[s], hv[c * S + s], sv[t][c]);
                    dc[s] = fmaf(gs[c], hv[c * S + s], dc[s]);
                }
            }
#pragma unroll
            for (int s = 0; s < S; ++s) sm.red[wave][cl][sg * V + t % TR * S + s] = dc[s];
            if (t % TR == TR - 1) {
                wave_lds_fence();
                join_channels<S, TR>(sm.red[wave], lane, [&](int tr, int n, float v) {
                    const int64_t tt = t0 + t - (TR - 1) + tr;
                    if (tt < p.T && n < p.N) part_c[tt * brow + n] = tt < len ? v : 0.f;
                });
                wave_lds_fence();
            }
        }
        // g in reverse and everything that depends on it
        float dxv[L][C], dd2[L][C];
#pragma unroll
        for (int t = L - 1; t >= 0; --t) {
            float x[2 * C], gs[C], bt[S], ct[S], db[S];
            __builtin_amdgcn_sched_barrier(0);
            lds_read<2 * C>(sm.x[wave][t][cl], x);
            lds_read<C>(sm.ds[wave][t][cl], gs);
            lds_read<S>(&sm.b[wave][0][t][sg * S], bt);
            lds_read<S>(&sm.b[wave][1][t][sg * S], ct);
#pragma unroll
            for (int s = 0; s < S; ++s) db[s] = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                dxv[t][c] = dd2[t][c] = 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const float gt = fmaf(ct[s], gs[c], gv[c * S + s]);
                    gv[c * S + s] = a[t][s][c] * gt;
                    const float q = gt * ah[t][s][c];
                    dxv[t][c] = fmaf(gt, bt[s], dxv[t][c]);
                    db[s] = fmaf(gt, x[C + c], db[s]);
                    dd2[t][c] = fmaf(q, A2[s][c], dd2[t][c]);
                    dA[s][c] = fmaf(q, x[c], dA[s][c]);
                }
            }
#pragma unroll
            for (int s = 0; s < S; ++s) sm.red[wave][cl][sg * V + t % TR * S + s] = db[s];
            if (t % TR == 0) {
                wave_lds_fence();
                join_channels<S, TR>(sm.red[wave], lane, [&](int tr, int n, float v) {
                    const int64_t tt = t0 + t + tr;
                    if (tt < p.T && n < p.N) part_b[tt * brow + n] = tt < len ? v : 0.f;
                });
                wave_lds_fence();
            }
        }
        float so[J][C], xo[J][C], ao[J][C];
        if (z) sg_join<L, C>(sv, so);
        sg_join<L, C>(dxv, xo);
        sg_join<L, C>(dd2, ao);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t t = t0 + 4 * j + sg;
            if (t < p.T) {
                const bool in = t < len;
                float o1[C], o2[C], o3[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float dx = xo[j][c];
                    o1[c] = in ? fmaf(dl[j][c], dx, skip[c] * ds[j][c]) : 0.f;
                    o2[c] = in ? fmaf(uu[j][c], dx, LN2 * ao[j][c]) * der[j][c] : 0.f;
                    if (in && c < nv) {
                        dskip[c] = fmaf(ds[j][c], uu[j][c], dskip[c]);
                        dbias[c] += o2[c];
                    }
                    if (z) {
                        const float sk = fmaf(skip[c], uu[j][c], so[j][c]);
                        o3[c] = in ? gy[j][c] * sk * dsilu(zz[j][c], sigmoid(zz[j][c])) : 0.f;
                    }
                }
                store_ch<T, C>(du + t * p.D, nv, vec, o1);
                store_ch<T, C>(ddelta + t * p.D, nv, vec, o2);
                if (z) store_ch<T, C>(dz + t * p.D, nv, vec, o3);
            }
        }
    }
#pragma unroll
    for (int f = 0; f < FPT; ++f)
        if (st_off[f] >= 0 && p.dh0) p.dh0[b * p.D * p.N + st_off[f]] = carry[f];
    // dA over the waves; dskip and ddelta_bias over the waves and lane rows too
    __syncthreads();
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
    __syncthreads();
    float *pa = p.part_a + b * (p.N + 2) * p.D;
#pragma unroll
    for (int f = 0; f < FPT; ++f) {
        const int i = tid + f * NT;
        if (st_off[f] >= 0) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) s += sm.s[w][i];
            const int64_t d = st_off[f] / p.N, n = st_off[f] - d * p.N;
            pa[n * p.D + d] = s;
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
    const auto kernel = scan_bwd_kernel<T, S, TL::C, TL::L, SCAN_NW>;
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
    if (D / G > 0x40000000 || G > 0x40000000) return MI_ERR_UNSUPPORTED;
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
