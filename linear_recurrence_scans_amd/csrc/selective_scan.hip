// selective_scan.hip -- the selective state-space scan: forward and the
// single-token step (the gradient is in selective_scan_bwd.hip).
//
// Per channel, state and step: the gate's exponent (mul), the gate (exp2), the
// input dl u Bm (mul), the state (fma), the output (fma), and for the carry a
// running product of gates applied to the state that entered the wave (mul) and
// its output (fma).  An exp2 takes two issue slots, so a state-step costs at
// least 8 slots of the vector ALU; with N = 16 states that is above the time of
// the 6 to 8 bytes a channel-step moves: the vector ALU is the bound.  All in all a
// state-step takes 12 slots of 4 cycles (softplus, the gate silu(z), conversions and
// joins the rest).  Measured (MI355X, N = 16, bf16): B = 8, T = 4096, D = 4096 740 us,
// the vector ALU busy for 82 % of it; B = 1, T = 8192, D = 4096 with z 191 us, 84 %.
// The step of 64 sequences, D = 4096: 8.3 us, 4.3 TB/s.
#include "checks.hpp"
#include "selective_scan.hpp"

namespace miscan {
namespace {

// SUM: the first kernel of a cut sequence, which only forms its segment's
// transform.
template <typename T, int S, int C, int L, int NW, int WPS, bool SUM>
__global__ __launch_bounds__(NW * 64, WPS) void scan_fwd_kernel(ScanArgs p) {
    constexpr int EL = S * C, J = L / 4, NP = 4 * S;
    constexpr int E = EL * 64;                      // states a tile
    constexpr int NT = NW * 64;
    constexpr int FPT = (E + NT - 1) / NT;          // folded states a thread
    constexpr int BPL = (L * NP + 63) / 64;         // Bm (Cm) values a lane loads
    constexpr int LB = L + 4;                       // row stride of Bm in LDS
    using LV = LaneVec<EL>;
    using QR = QuadRow<S>;
    constexpr int NB = QR::NB;
    using PC = Pack<T, C>;
    using raw_t = typename PC::raw_t;
    using one_t = typename Pack<T, 1>::raw_t;
    __shared__ __align__(16) float sm_x[NW][L][16][2 * C];   // dl, dl u
    __shared__ __align__(16) float sm_b[NW][NP][LB];         // Bm by state
    __shared__ __align__(16) float sm_c[NW][L][NP];          // Cm by step
    __shared__ __align__(16) float sm_s[NW][E], sm_p[NW][E];
    const int item = xcd_item(p.n_items);
    if (item >= p.n_items) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int sg = lane >> 4, cl = lane & 15;
    const Item it(item, p);
    const int tile = it.tile, g = it.g, seg = it.seg;
    const int64_t b = it.b;
    const int64_t t_first = seg * p.seg, t_last = t_first + p.seg < p.T ? t_first + p.seg : p.T;
    const int ch0 = tile * 16 * C;                  // first channel of the tile inside its group
    const int64_t d0 = (int64_t)g * p.per + ch0;
    const int nch = p.per - ch0 < 16 * C ? p.per - ch0 : 16 * C;
    const int nv = nch - cl * C < 0 ? 0 : nch - cl * C > C ? C : nch - cl * C;
    const int64_t len = seq_len(p.lengths, b, p.T);
    const bool whole = C == 1 || p.vec;             // rows go by whole vectors
    float A2[S][C], skip[C], bias[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t d = d0 + cl * C + c;
        const bool ok = c < nv;
        skip[c] = ok && p.skip ? p.skip[d] : 0.f;
        bias[c] = ok && p.delta_bias ? p.delta_bias[d] : 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int n = sg * S + s;
            A2[s][c] = ok && n < p.N ? gate_base(p.A[d * p.N + n]) : 0.f;
        }
    }
    // folded states: thread tid carries positions tid, tid + NT, ... of the tile
    float carry[FPT], prod[FPT];
    int st_off[FPT];  // offset from the tile's first state, or -1
    const int64_t st_base = b * p.D * p.N + d0 * p.N;
#pragma unroll
    for (int f = 0; f < FPT; ++f) {
        const int i = tid + f * NT;
        int ln, e;
        LV::where(i < E ? i : 0, &ln, &e);
        const int n = (ln >> 4) * S + e % S, ch = (ln & 15) * C + e / S;
        st_off[f] = i < E && n < p.N && ch < nch ? ch * (int)p.N + n : -1;
        carry[f] = !SUM && st_off[f] >= 0 && p.h0 ? p.h0[st_base + st_off[f]] : 0.f;
        if (!SUM && st_off[f] >= 0) {
            const float *v = p.seg_v + st_base + st_off[f], *q = p.seg_p + st_base + st_off[f];
#pragma unroll 4
            for (int k = 0; k < seg; ++k)
                carry[f] = carry_through(q[k * p.B * p.D * p.N], carry[f], v[k * p.B * p.D * p.N]);
        }
        prod[f] = 1.f;
    }
    // a lane's rows: steps sg, 4 + sg, ... of the wave's, as byte offsets from the wave's first
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
    raw_t ur[J], dr[J], zr[J];
    one_t br[BPL], cr[BPL];

    // the wave's rows of the block in which its steps start at t0
    const auto load = [&](int64_t t0) {
        const int64_t left = steps_left<L>(t0, len);
        load_rows<T, C, J>(make_rows(static_cast<const T *>(p.u) + row0 + t0 * p.D, left * row), voff, nv, whole, ur);
        load_rows<T, C, J>(make_rows(static_cast<const T *>(p.delta) + row0 + t0 * p.D, left * row), voff, nv, whole,
                           dr);
        if (!SUM && p.z)
            load_rows<T, C, J>(make_rows(static_cast<const T *>(p.z) + row0 + t0 * p.D, left * row), voff, nv, whole,
                               zr);
        const rsrc_t rb = make_rows(static_cast<const T *>(p.Bm) + b0 + t0 * brow, left * brow * (int64_t)sizeof(T));
        const rsrc_t rc = make_rows(static_cast<const T *>(p.Cm) + b0 + t0 * brow, left * brow * (int64_t)sizeof(T));
#pragma unroll
        for (int i = 0; i < BPL; ++i) {
            br[i] = buf_read<T, 1>(rb, boff[i]);
            if (!SUM) cr[i] = buf_read<T, 1>(rc, boff[i]);
        }
    };

    // blocks past the sequence's end leave the state and have zero rows
    const int64_t t_end = len < t_last ? (len < t_first ? t_first : (len - t_first + NW * L - 1) / (NW * L) * (NW * L) + t_first)
                                       : t_last;
    load(t_first + wave * L);
    for (int64_t tb = t_first; tb < t_end; tb += NW * L) {
        const int64_t t0 = tb + wave * L;
        const int left = steps_left<L>(t0, len);
        // this wave's rows: dl and dl u by the lanes that own them
        raw_t uk[J], zk[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float uu[C], dd[C], o[2 * C];
            PC::unpack(ur[j], uu);
            PC::unpack(dr[j], dd);
            uk[j] = ur[j];
            zk[j] = zr[j];
            const bool in = 4 * j + sg < left;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float r = gate_rate(dd[c] + bias[c], p.softplus, nullptr);
                o[c] = in ? r : 0.f;
                o[C + c] = o[c] * uu[c];
            }
#pragma unroll
            for (int i = 0; i < 2 * C; ++i) sm_x[wave][4 * j + sg][cl][i] = o[i];
        }
#pragma unroll
        for (int i = 0; i < BPL; ++i) {
            const int q = lane + 64 * i, t = q / NP, n = q % NP;
            if (L * NP % 64 == 0 || q < L * NP) {
                Pack<T, 1>::unpack(br[i], &sm_b[wave][n][t]);
                if (!SUM) Pack<T, 1>::unpack(cr[i], &sm_c[wave][t][n]);
            }
        }
        if (tb + NW * L < t_end) load(t0 + NW * L);
        wave_lds_sync();
        // the wave's steps from a zero state
        float a[L][S][C], h[S][C], yl[L][C], sum[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            sum[c] = 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s) h[s][c] = 0.f;
        }
        const int n0 = QR::first(lane);
#pragma unroll
        for (int tq = 0; tq < L; tq += 4) {
            float bq[NB][4];
#pragma unroll
            for (int i = 0; i < NB; ++i) lds_read<4>(&sm_b[wave][n0 + 4 * i][tq], bq[i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = tq + k;
                __builtin_amdgcn_sched_barrier(0);
                float dx[2 * C], bt[NB], ct[S];
                lds_read<2 * C>(sm_x[wave][t][cl], dx);
                if constexpr (!SUM) lds_read<S>(&sm_c[wave][t][sg * S], ct);
#pragma unroll
                for (int i = 0; i < NB; ++i) bt[i] = bq[i][k];
#pragma unroll
                for (int c = 0; c < C; ++c) { sum[c] += dx[c]; yl[t][c] = 0.f; }
                for_each<S>([&](auto si) {
                    constexpr int s = decltype(si)::value;
                    const float bs = QR::template get<s>(bt);
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const float gate = __builtin_amdgcn_exp2f(dx[c] * A2[s][c]);
                        const float x = bs * dx[C + c];
                        h[s][c] = t == 0 ? x : fmaf(gate, h[s][c], x);
                        if constexpr (!SUM) {
                            a[t][s][c] = gate;
                            yl[t][c] = fmaf(ct[s], h[s][c], yl[t][c]);
                        }
                    }
                });
                if constexpr (!SUM) {
                    pin(yl[t]);
                } else {
#pragma unroll
                    for (int s = 0; s < S; ++s) pin(h[s]);
                }
            }
        }
        float hv[EL], pv[EL];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int s = 0; s < S; ++s) {
                hv[c * S + s] = h[s][c];
                pv[c * S + s] = SUM ? root_product(sum[c] * A2[s][c]) : __builtin_amdgcn_exp2f(sum[c] * A2[s][c]);
            }
        LV::write(sm_s[wave], lane, hv);
        LV::write(sm_p[wave], lane, pv);
        wg_lds_sync();
#pragma unroll
        for (int f = 0; f < FPT; ++f) {
            const int i = tid + f * NT;
            if (i < E) {
                float c = carry[f], sv[NW], pw[NW];
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    sv[w] = sm_s[w][i];
                    pw[w] = sm_p[w][i];
                }
                if constexpr (SUM) {
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        prod[f] = join_roots(prod[f], pw[w]);
                        c = carry_through(pw[w], c, sv[w]);
                    }
                } else {
                    // state v enters wave w
                    const auto enter = [&](int w, float v) {
                        if ((w * L) % scan_block_of<S>() % (NW * L) == 0 && (tb + w * L) % scan_block_of<S>() == 0 &&
                            p.states && st_off[f] >= 0 && tb + w * L < p.T) {
                            const int64_t blk = (tb + w * L) / scan_block_of<S>();
                            const int64_t n_blk = (p.T + scan_block_of<S>() - 1) / scan_block_of<S>();
                            p.states[(b * n_blk + blk) * p.D * p.N + d0 * p.N + st_off[f]] = v;
                        }
                        sm_s[w][i] = v;
                    };
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        enter(w, c);
                        c = fmaf(pw[w], c, sv[w]);
                    }
                    // a product out of range: step by step, from the first wave that a value
                    // which is not finite enters (so do all after it)
                    const bool bad = !__builtin_isfinite(c);
                    if (__builtin_expect(__any(bad), 0) && bad) {
                        int ln, e;
                        LV::where(i, &ln, &e);
                        const int n = (ln >> 4) * S + e % S, q = e / S;
                        const float a2 = st_off[f] >= 0 ? gate_base(p.A[d0 * p.N + st_off[f]]) : 0.f;
                        c = carry[f];
#pragma unroll 1
                        for (int w = 0; w < NW; ++w) {
                            const float v = sm_s[w][i];
                            if (__builtin_isfinite(v)) c = v;
                            else enter(w, c);
#pragma unroll 1
                            for (int t = 0; t < L; ++t) {
                                const float *x = sm_x[w][t][ln & 15];
                                c = fmaf(__builtin_amdgcn_exp2f(x[q] * a2), c, sm_b[w][n][t] * x[C + q]);
                            }
                        }
                    }
                }
                carry[f] = c;
            }
        }
        wg_lds_sync();
        if constexpr (SUM) continue;
        // the state that entered the wave, carried through its gates
        LV::read(sm_s[wave], lane, hv);
#pragma unroll
        for (int t = 0; t < L; ++t) {
            __builtin_amdgcn_sched_barrier(0);
            float ct[S];
            lds_read<S>(&sm_c[wave][t][sg * S], ct);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    hv[c * S + s] *= a[t][s][c];
                    yl[t][c] = fmaf(ct[s], hv[c * S + s], yl[t][c]);
                }
            pin(yl[t]);
        }
        float out[J][C];
        sg_join<L, C>(yl, out);
        char *y = reinterpret_cast<char *>(static_cast<T *>(p.y) + row0 + t0 * p.D);
        const int rows = steps_left<L>(t0, p.T);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float uu[C], zz[C], o[C];
            PC::unpack(uk[j], uu);
            PC::unpack(zk[j], zz);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                o[c] = fmaf(skip[c], uu[c], out[j][c]);
                if (p.z) o[c] *= silu(zz[c]);
                if (4 * j + sg >= left) o[c] = 0.f;
            }
            if (4 * j + sg < rows) store_ch<T, C>(y + voff[j], nv, whole, o);
        }
    }
    if constexpr (SUM) {
#pragma unroll
        for (int f = 0; f < FPT; ++f)
            if (st_off[f] >= 0) {
                const int64_t at = seg * p.B * p.D * p.N + st_base + st_off[f];
                p.seg_v[at] = carry[f];
                p.seg_p[at] = prod[f];
            }
        return;
    }
    const float zero[C] = {};
    for (int64_t tb = t_end; tb < t_last; tb += NW * L) {
        const int64_t t0 = tb + wave * L;
        char *y = reinterpret_cast<char *>(static_cast<T *>(p.y) + row0 + t0 * p.D);
        const int rows = steps_left<L>(t0, p.T);
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (4 * j + sg < rows) store_ch<T, C>(y + voff[j], nv, whole, zero);
    }
    if (p.states) {
        constexpr int64_t BLK = scan_block_of<S>();
        const int64_t n_blk = (p.T + BLK - 1) / BLK;
        for (int64_t k = (t_end + BLK - 1) / BLK; k * BLK < t_last; ++k)
#pragma unroll
            for (int f = 0; f < FPT; ++f)
                if (st_off[f] >= 0) p.states[(b * n_blk + k) * p.D * p.N + d0 * p.N + st_off[f]] = carry[f];
    }
    if (p.hT && seg == p.n_seg - 1)
#pragma unroll
        for (int f = 0; f < FPT; ++f)
            if (st_off[f] >= 0) p.hT[st_base + st_off[f]] = carry[f];
}

// One token: a lane owns up to four states of a channel, LQ lanes a channel, a
// workgroup 256 / LQ channels of one sequence.  The state is read and written
// once, which is nearly all the traffic: the bound is HBM.  QUAD: rows of whole,
// aligned quads.
template <typename T, int LQ, bool QUAD>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanArgs p, int wg_row) {
    const int64_t b = blockIdx.x / wg_row;
    const int c = (int)(blockIdx.x - (int)b * wg_row) * (256 / LQ) + (int)threadIdx.x / LQ;
    const int q = (int)threadIdx.x % LQ;
    const bool live = c < p.D;
    const int64_t d = live ? c : 0, chan = b * p.D + d;
    const int N = (int)p.N, n0 = 4 * q;
    const int nv = !live ? 0 : N - n0 < 0 ? 0 : N - n0 > 4 ? 4 : N - n0;
    const int64_t brow = (b * p.G + (p.G > 1 ? (int)d / p.per : 0)) * N + n0;
    float h[4], A[4], Bv[4], Cv[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) h[s] = A[s] = Bv[s] = Cv[s] = 0.f;
    const float *hp = p.h0 + chan * N + n0, *ap = p.A + d * N + n0;
    const T *bp = static_cast<const T *>(p.Bm) + brow, *cp = static_cast<const T *>(p.Cm) + brow;
    if (QUAD) {
        if (nv > 0) {
            Pack<float, 4>::unpack(load_vec<float, 4>(hp), h);
            Pack<float, 4>::unpack(load_vec<float, 4>(ap), A);
            Pack<T, 4>::unpack(load_vec<T, 4>(bp), Bv);
            Pack<T, 4>::unpack(load_vec<T, 4>(cp), Cv);
        }
    } else {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            if (s < nv) {
                h[s] = hp[s];
                A[s] = ap[s];
                Bv[s] = ld1(bp + s);
                Cv[s] = ld1(cp + s);
            }
    }
    const float uu = ld1(static_cast<const T *>(p.u) + chan);
    const float raw = ld1(static_cast<const T *>(p.delta) + chan) + (p.delta_bias ? p.delta_bias[d] : 0.f);
    const float zz = p.z ? ld1(static_cast<const T *>(p.z) + chan) : 0.f;
    const float dl = gate_rate(raw, p.softplus, nullptr);
    float acc = 0.f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        h[s] = fmaf(__builtin_amdgcn_exp2f(dl * gate_base(A[s])), h[s], dl * uu * Bv[s]);
        acc = fmaf(Cv[s], h[s], acc);
    }
    float *ho = p.hT + chan * N + n0;
    if (QUAD) {
        if (nv > 0) *reinterpret_cast<f32x4 *>(ho) = Pack<float, 4>::pack(h);
    } else {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            if (s < nv) ho[s] = h[s];
    }
#pragma unroll
    for (int m = 1; m < LQ; m *= 2) acc += __shfl_xor(acc, m);
    if (live && q == 0) {
        if (p.skip) acc = fmaf(p.skip[d], uu, acc);
        if (p.z) acc *= silu(zz);
        st1(static_cast<T *>(p.y) + chan, acc);
    }
}

template <typename T, int LQ>
mi_status launch_step(const ScanArgs &a, bool quad, hipStream_t s) {
    const int64_t wg_row = (a.D + 256 / LQ - 1) / (256 / LQ);
    int64_t grid;
    if (!mul_ok(a.B, wg_row, 1, 1, &grid) || !launch_fits(grid, 256)) return MI_ERR_UNSUPPORTED;
    const dim3 gd((unsigned)grid), bd(256);
    if (quad) hipLaunchKernelGGL((scan_step_kernel<T, LQ, true>), gd, bd, 0, s, a, (int)wg_row);
    else hipLaunchKernelGGL((scan_step_kernel<T, LQ, false>), gd, bd, 0, s, a, (int)wg_row);
    return launch_status();
}
template <typename T>
mi_status launch_step_t(const ScanArgs &a, hipStream_t s) {
    const auto at = [](const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    const bool quad = a.N % 4 == 0 && at(a.h0, 16) && at(a.hT, 16) && at(a.A, 16) && at(a.Bm, 4 * sizeof(T)) &&
                      at(a.Cm, 4 * sizeof(T));
    if (a.N <= 4) return launch_step<T, 1>(a, quad, s);
    if (a.N <= 8) return launch_step<T, 2>(a, quad, s);
    if (a.N <= 16) return launch_step<T, 4>(a, quad, s);
    if (a.N <= 32) return launch_step<T, 8>(a, quad, s);
    return launch_step<T, 16>(a, quad, s);
}

template <typename T, int S, int C, int L, int NW, int WPS, bool CUT>
mi_status launch_tile(ScanArgs a, int64_t n_seg, hipStream_t s) {
    a.tiles = (a.per + 16 * C - 1) / (16 * C);
    int64_t items;
    if (!mul_ok(a.B, a.G, a.tiles, n_seg, &items) || !launch_fits(items + 7, NW * 64)) return MI_ERR_UNSUPPORTED;
    a.n_seg = (int)n_seg;
    a.seg = (a.T + NW * L * n_seg - 1) / (NW * L * n_seg) * (NW * L);
    if constexpr (CUT)
        if (n_seg > 1) {
            a.n_items = (int)(items / n_seg * (n_seg - 1));  // nothing needs the last segment's transform
            hipLaunchKernelGGL((scan_fwd_kernel<T, S, C, L, NW, WPS, true>), dim3(xcd_grid(a.n_items)),
                               dim3(NW * 64), 0, s, a);
            const mi_status st = launch_status();
            if (st != MI_OK) return st;
        }
    a.n_items = (int)items;
    hipLaunchKernelGGL((scan_fwd_kernel<T, S, C, L, NW, WPS, false>), dim3(xcd_grid(a.n_items)), dim3(NW * 64), 0, s,
                       a);
    return launch_status();
}

// How a call is cut, by the number of workgroups that its channel tiles make.  Times in
// us, bf16 with z, n wide tiles (two channels a lane, one for N > 16):
//  - 640 or more wide tiles: workgroups of 4 waves at 3 waves a SIMD, which
//    overlap each other's folds;
//  - fewer: narrow tiles (one channel a lane) of 16 waves, while those make at
//    least 192 workgroups: twice the workgroups, four times the waves.  (N > 32, whose
//    tiles are narrow already and whose LDS holds 8 waves: 8 waves.)
//        N                     4          8          16         32         64
//        wide / narrow
//        n = 256, T = 2048     102 / 65   132 / 83   178 / 110  153 / 104  305 / 210
//        n = 512, T = 2048     115 / 125  159 / 156  224 / 205  202 / 196  405 / 410
//        n = 640, T = 2048     141 / 177  193 / 209  289 / 262  260 / 289  642 / 611
//        n = 1024, T = 1024    108 / 137  125 / 168  203 / 222  182 / 205  399 / 421
//  - fewer still: segments of the sequence, as many as the CUs hold at once (3
//    workgroups of 4 waves, 2 for N > 32): more would run in a second turn.  B = 1,
//    T = 4096, N = 16: n = 60 100 us in 12 segments and 111 in 13, n = 90 137 in 8 and 156
//    in 9.  Against narrow tiles, n = 64: N = 4 53 and 64, N = 16 103 and 101, N = 32 98 and
//    187, N = 64 192 and 403 us.  At most 4 sqrt(blocks) of them, a block being 4 waves'
//    steps: each folds all that come before it.  B = 1, T = 8192, N = 16, 256 blocks: D =
//    64 101 us in 256 segments, 47 in 128, 41 in 64 and 52 in 32; N = 64, 512 blocks, D =
//    64 454 in 256, 138 in 128, 72 in 64; T = 65536, D = 16 183 in 683, 100 in 128.
enum FwdCut { FWD_MANY, FWD_NARROW, FWD_SEGMENTS };
struct FwdPlan {
    FwdCut cut;
    int64_t n_seg;
};
constexpr int fwd_wps(int S) { return S == 16 ? 2 : 3; }  // waves a SIMD of wide tiles
inline int64_t fwd_slots(int S, int64_t n) { return (S == 16 && n > 64 ? 2 : 1) * 256 * fwd_wps(S); }
template <int S>
FwdPlan fwd_plan(int64_t B, int64_t G, int64_t per, int64_t T) {
    constexpr int C = FwdTile<S>::C, L = FwdTile<S>::L;
    const int64_t n = B * G * ((per + 16 * C - 1) / (16 * C)), narrow = B * G * ((per + 15) / 16);
    if (n >= 640) return {FWD_MANY, 1};
    if (narrow >= 192) return {FWD_NARROW, 1};
    const int64_t blocks = (T + 4 * L - 1) / (4 * L), fill = fwd_slots(S, n) / n;
    const int64_t deep = (int64_t)(4.0 * sqrt((double)blocks));
    const int64_t want = fill < deep ? fill : deep < 1 ? 1 : deep;
    const int64_t seg = (blocks + want - 1) / want;  // blocks a segment
    // (a second launch costs the host about two blocks' time, its segments two more)
    return {FWD_SEGMENTS, blocks < 8 ? 1 : (blocks + seg - 1) / seg};
}
int64_t fwd_segments(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    switch (scan_s(N)) {
        case 1: return fwd_plan<1>(B, G, D / G, T).n_seg;
        case 2: return fwd_plan<2>(B, G, D / G, T).n_seg;
        case 4: return fwd_plan<4>(B, G, D / G, T).n_seg;
        case 8: return fwd_plan<8>(B, G, D / G, T).n_seg;
    }
    return fwd_plan<16>(B, G, D / G, T).n_seg;
}

template <typename T, int S>
mi_status launch_fwd(const ScanArgs &a, hipStream_t s) {
    constexpr int C = FwdTile<S>::C, L = FwdTile<S>::L;
    constexpr int WPS = fwd_wps(S);
    constexpr int LN = S >= 8 ? 4 : S >= 2 ? 8 : 16;  // narrow: at most 32 gates a lane, 128 registers
    const FwdPlan q = fwd_plan<S>(a.B, a.G, a.per, a.T);
    if (q.cut == FWD_NARROW) return launch_tile<T, S, 1, LN, S == 16 ? 8 : 16, S == 16 ? 2 : 4, false>(a, 1, s);
    return launch_tile<T, S, C, L, 4, WPS, true>(a, q.n_seg, s);
}
template <typename T>
mi_status launch_fwd_t(const ScanArgs &a, hipStream_t s) {
    switch (scan_s(a.N)) {
        case 1: return launch_fwd<T, 1>(a, s);
        case 2: return launch_fwd<T, 2>(a, s);
        case 4: return launch_fwd<T, 4>(a, s);
        case 8: return launch_fwd<T, 8>(a, s);
    }
    return launch_fwd<T, 16>(a, s);
}

}  // namespace

mi_status check_scan(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, mi_dtype dt, ScanSizes *s) {
    if (B < 0 || T < 0 || D < 0 || G < 1 || N < 0) return MI_ERR_INVALID_ARG;
    if (!dtype_known(dt) || N < 1 || N > 64) return MI_ERR_UNSUPPORTED;
    if (D % G != 0) return MI_ERR_INVALID_ARG;
    const int64_t es = (int64_t)elem_size(dt);
    int64_t gn;
    if (!mul_ok(B, T, D, es, &s->x) || !mul_ok(G, N, es, 1, &gn) || !mul_ok(B, T, gn, 1, &s->bc) ||
        !mul_ok(B, D, N, 4, &s->h) || !mul_ok(D, N, 4, 1, &s->a))
        return MI_ERR_INVALID_ARG;
    s->d = D * 4;
    const int64_t blk = scan_block(N);
    if (!mul_ok(s->h, T / blk + (T % blk != 0), 1, 1, &s->states)) return MI_ERR_INVALID_ARG;
    return MI_OK;
}

// Rows may be read C channels at a time: groups of even width, even row starts,
// pointers aligned to the pair.
bool scan_vec(const ScanArgs &a, mi_dtype dt) {
    const Buf b[8] = {{a.u, 1}, {a.delta, 1}, {a.z, 1}, {a.y, 1}, {a.dy, 1}, {a.du, 1}, {a.ddelta, 1}, {a.dz, 1}};
    return a.D % 2 == 0 && a.per % 2 == 0 && pick_vec(2, elem_size(dt), b, 8) == 2;
}

}  // namespace miscan

using namespace miscan;

extern "C" {

int64_t mi_selective_scan_block(int64_t N) { return N < 1 || N > 64 ? 0 : scan_block(N); }

size_t mi_selective_scan_fwd_workspace(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, mi_dtype dt) {
    ScanSizes s;
    if (check_scan(B, T, D, G, N, dt, &s) != MI_OK || B == 0 || T == 0 || D == 0) return 0;
    const int64_t n = fwd_segments(B, T, D, G, N);
    int64_t bytes;
    return n > 1 && mul_ok(s.h, n, 2, 1, &bytes) ? (size_t)bytes : 0;
}

mi_status mi_selective_scan_fwd(const void *u, const void *delta, const float *A, const void *Bm, const void *Cm,
                                const float *skip, const void *z, const float *delta_bias, const float *h0,
                                const int32_t *lengths, void *y, float *hT, float *states, int64_t B, int64_t T,
                                int64_t D, int64_t G, int64_t N, int softplus_on, mi_dtype dt, void *ws,
                                size_t ws_bytes, hipStream_t stream) {
    ScanSizes s;
    mi_status st = check_scan(B, T, D, G, N, dt, &s);
    if (st != MI_OK) return st;
    if (B == 0 || D == 0 || (T == 0 && hT == nullptr)) return MI_OK;
    const size_t es = elem_size(dt);
    BufList in, out;
    in.need(u, s.x, es).need(delta, s.x, es).need(A, s.a, 4).need(Bm, s.bc, es).need(Cm, s.bc, es);
    in.opt(skip, s.d, 4).opt(z, s.x, es).opt(delta_bias, s.d, 4).opt(h0, s.h, 4).opt(lengths, B * 4, 4);
    out.need(y, s.x, es).opt(hT, s.h, 4).opt(states, s.states, 4);
    if ((st = check_lists(in, out)) != MI_OK) return st;
    ScanArgs a{};
    a.u = u; a.delta = delta; a.z = z; a.Bm = Bm; a.Cm = Cm; a.A = A; a.skip = skip; a.delta_bias = delta_bias;
    a.h0 = h0; a.lengths = lengths; a.y = y; a.hT = hT; a.states = states;
    a.B = B; a.T = T; a.D = D; a.N = N; a.softplus = softplus_on != 0;
    const size_t need = mi_selective_scan_fwd_workspace(B, T, D, G, N, dt);
    if (need > 0) {
        if ((st = check_ws_lists(ws, ws_bytes, need, in, out)) != MI_OK) return st;
        a.seg_v = static_cast<float *>(ws);
        a.seg_p = a.seg_v + need / 8;
    }
    if (D > SCAN_MAX_D || G * N > SCAN_MAX_D) return MI_ERR_UNSUPPORTED;
    a.G = (int)G; a.per = (int)(D / G);
    a.vec = scan_vec(a, dt);
    if (dt == MI_F32) return launch_fwd_t<float>(a, stream);
    if (dt == MI_BF16) return launch_fwd_t<bf16_t>(a, stream);
    return launch_fwd_t<f16_t>(a, stream);
}

mi_status mi_selective_scan_step(const void *u, const void *delta, const float *A, const void *Bm, const void *Cm,
                                 const float *h, const float *skip, const void *z, const float *delta_bias, void *y,
                                 float *h_out, int64_t B, int64_t D, int64_t G, int64_t N, int softplus_on,
                                 mi_dtype dt, hipStream_t stream) {
    ScanSizes s;
    mi_status st = check_scan(B, 1, D, G, N, dt, &s);
    if (st != MI_OK || B == 0 || D == 0) return st;
    const size_t es = elem_size(dt);
    BufList in, out;
    in.need(u, s.x, es).need(delta, s.x, es).need(A, s.a, 4).need(Bm, s.bc, es).need(Cm, s.bc, es);
    in.opt(skip, s.d, 4).opt(z, s.x, es).opt(delta_bias, s.d, 4);
    if (h != h_out) in.need(h, s.h, 4);  // in place: the state is checked as an output
    out.need(y, s.x, es).need(h_out, s.h, 4);
    if ((st = check_lists(in, out)) != MI_OK) return st;
    ScanArgs a{};
    a.u = u; a.delta = delta; a.z = z; a.Bm = Bm; a.Cm = Cm; a.A = A; a.skip = skip; a.delta_bias = delta_bias;
    a.h0 = h; a.y = y; a.hT = h_out;
    a.B = B; a.T = 1; a.D = D; a.N = N; a.softplus = softplus_on != 0;
    if (D > SCAN_MAX_D || G * N > SCAN_MAX_D) return MI_ERR_UNSUPPORTED;
    a.G = (int)G; a.per = (int)(D / G);
    if (dt == MI_F32) return launch_step_t<float>(a, stream);
    if (dt == MI_BF16) return launch_step_t<bf16_t>(a, stream);
    return launch_step_t<f16_t>(a, stream);
}

}  // extern "C"
