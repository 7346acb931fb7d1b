// group_norm.hip -- group norm over the channels of each row (channels last),
// with an activation or a gate, and its gradient.
//
// A team of TEAM lanes holds one group of one row in registers (NV vectors of
// VEC elements a lane), so a row is read once; mean and variance are two team
// sums (the variance about the mean, no cancellation).  A lane keeps its
// channels' parameters, and in the backward their gradients' sums, in registers
// over all the rows its workgroup walks.  The bound is HBM: forward 2 to 3,
// backward 3 to 5 tensors moved once.  Measured (MI355X, 16384 x 4096, gated): bf16 in
// 32 groups forward 75 us (5.4 TB/s), backward 142 (4.7 TB/s) and its sums 6; bf16 in one
// group forward 69 (5.9 TB/s), both 240; fp32 in 32 groups 176 (4.6 TB/s) and 459, in one
// group 153 (5.3 TB/s) and 466.
#include "block_ops.hpp"
#include "checks.hpp"

namespace miscan {
namespace {

struct NormArgs {
    const void *x, *z, *dy;
    const float *w, *bias;
    void *y, *dx, *dz;
    float *part;       // (parts, 2, D) partial dw, dbias
    int64_t R, D;
    int64_t rows;      // rows a workgroup walks
    int G, dg;         // groups, channels a group
    int gps, n_slices; // groups side by side in a wave; slices of them
    float eps, inv_dg;
    int centered, act;
};

// Sum over a team, the same value in all its lanes.  Teams of 256 are whole
// workgroups; `sm` then holds one value a wave and is free again on return.
template <int TEAM, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*sm)[4]) {
#pragma unroll
    for (int m = 1; m < (TEAM < 64 ? TEAM : 64); m *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], m);
    if constexpr (TEAM == 256) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) sm[i][wave] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = (sm[i][0] + sm[i][1]) + (sm[i][2] + sm[i][3]);
    }
}

// Place of a thread: its group's first channel, its lane in the team, the row
// it starts with and the rows between two of its own.
struct Place {
    int64_t c0;
    int q;
    int64_t row, step;
    bool ok;
};
template <int TEAM>
__device__ __forceinline__ Place place(const NormArgs &p, int slice, int part) {
    Place o;
    const int tid = threadIdx.x;
    const int64_t first = (int64_t)part * p.rows;
    if constexpr (TEAM == 256) {
        o.q = tid;
        o.c0 = (int64_t)slice * p.dg;
        o.row = first;
        o.step = 1;
        o.ok = true;
    } else {
        const int lane = tid & 63, wave = tid >> 6, team = lane / TEAM;
        const int grp = slice * p.gps + team % p.gps, per = 64 / TEAM / p.gps;
        o.q = lane % TEAM;
        o.c0 = (int64_t)grp * p.dg;
        o.row = first + wave * per + team / p.gps;
        o.step = 4 * per;
        o.ok = grp < p.G;
    }
    return o;
}

template <typename T, int VEC, int NV, int TEAM>
struct Held {
    using PK = Pack<T, VEC>;
    // element index of vector j of team lane q inside the group
    static __device__ __forceinline__ int at(int q, int j) { return (j * TEAM + q) * VEC; }
    static __device__ __forceinline__ void load(const T *p, int q, int dg, bool ok, float (&f)[NV][VEC]) {
        typename PK::raw_t raw[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            raw[j] = splat<T, VEC>(0.f);
            if (ok && at(q, j) < dg) raw[j] = load_vec<T, VEC>(p + at(q, j));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) PK::unpack(raw[j], f[j]);
    }
    static __device__ __forceinline__ void params(const float *p, int q, int dg, bool ok, float dflt,
                                                  float (&f)[NV][VEC]) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < VEC; ++v) f[j][v] = p != nullptr && ok && at(q, j) < dg ? p[at(q, j) + v] : dflt;
    }
};

// x becomes xh; returns 1 / sqrt(var + eps).
template <int VEC, int NV, int TEAM>
__device__ __forceinline__ float normalise(const NormArgs &p, int q, float (&x)[NV][VEC], float (*sm)[4]) {
    float s[1] = {0.f};
    if (p.centered) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < VEC; ++v) s[0] += x[j][v];
        team_sum<TEAM>(s, sm);
        const float mean = s[0] * p.inv_dg;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < VEC; ++v) x[j][v] = (j * TEAM + q) * VEC < p.dg ? x[j][v] - mean : 0.f;
    }
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int v = 0; v < VEC; ++v) s[0] = fmaf(x[j][v], x[j][v], s[0]);
    team_sum<TEAM>(s, sm);
    const float rstd = __builtin_amdgcn_rsqf(fmaf(s[0], p.inv_dg, p.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int v = 0; v < VEC; ++v) x[j][v] *= rstd;
    return rstd;
}

template <typename T, int VEC, int NV, int TEAM>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs p) {
    using H = Held<T, VEC, NV, TEAM>;
    __shared__ float sm[2][4];
    const int slice = blockIdx.x % p.n_slices, part = blockIdx.x / p.n_slices;
    const Place o = place<TEAM>(p, slice, part);
    float w[NV][VEC], bias[NV][VEC];
    H::params(p.w ? p.w + o.c0 : nullptr, o.q, p.dg, o.ok, 1.f, w);
    H::params(p.bias ? p.bias + o.c0 : nullptr, o.q, p.dg, o.ok, 0.f, bias);
    const int64_t last = (int64_t)(part + 1) * p.rows < p.R ? (int64_t)(part + 1) * p.rows : p.R;
    // every lane of a wave runs as often as its first row does: the team sums
    // need whole waves
    const int64_t turns = (last - (int64_t)part * p.rows + o.step - 1) / o.step;
    for (int64_t i = 0; i < turns; ++i) {
        const int64_t r = o.row + i * o.step;
        const bool ok = o.ok && r < last;
        const int64_t base = r * p.D + o.c0;
        float x[NV][VEC], z[NV][VEC];
        H::load(static_cast<const T *>(p.x) + base, o.q, p.dg, ok, x);
        if (p.z) H::load(static_cast<const T *>(p.z) + base, o.q, p.dg, ok, z);
        normalise<VEC, NV, TEAM>(p, o.q, x, sm);
        T *y = static_cast<T *>(p.y) + base;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float f[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                f[v] = fmaf(x[j][v], w[j][v], bias[j][v]);
                if (p.act == MI_ACT_SILU) f[v] = silu(f[v]);
                if (p.z) f[v] *= silu(z[j][v]);
            }
            if (ok && H::at(o.q, j) < p.dg) store_vec<T, VEC>(y + H::at(o.q, j), Pack<T, VEC>::pack(f));
        }
    }
}

template <typename T, int VEC, int NV, int TEAM>
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormArgs p) {
    using H = Held<T, VEC, NV, TEAM>;
    __shared__ float sm[2][4];
    __shared__ float acc[2][4][64];
    const int slice = blockIdx.x % p.n_slices, part = blockIdx.x / p.n_slices;
    const Place o = place<TEAM>(p, slice, part);
    float w[NV][VEC], bias[NV][VEC], dw[NV][VEC], db[NV][VEC];
    H::params(p.w ? p.w + o.c0 : nullptr, o.q, p.dg, o.ok, 1.f, w);
    H::params(p.bias ? p.bias + o.c0 : nullptr, o.q, p.dg, o.ok, 0.f, bias);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int v = 0; v < VEC; ++v) dw[j][v] = db[j][v] = 0.f;
    const int64_t last = (int64_t)(part + 1) * p.rows < p.R ? (int64_t)(part + 1) * p.rows : p.R;
    const int64_t turns = (last - (int64_t)part * p.rows + o.step - 1) / o.step;
    for (int64_t i = 0; i < turns; ++i) {
        const int64_t r = o.row + i * o.step;
        const bool ok = o.ok && r < last;
        const int64_t base = r * p.D + o.c0;
        float x[NV][VEC], z[NV][VEC], g[NV][VEC];
        H::load(static_cast<const T *>(p.x) + base, o.q, p.dg, ok, x);
        H::load(static_cast<const T *>(p.dy) + base, o.q, p.dg, ok, g);
        if (p.z) H::load(static_cast<const T *>(p.z) + base, o.q, p.dg, ok, z);
        const float rstd = normalise<VEC, NV, TEAM>(p, o.q, x, sm);
        float c[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float pv = fmaf(x[j][v], w[j][v], bias[j][v]);
                float dp = g[j][v];
                if (p.z) {
                    const float sig = sigmoid(z[j][v]);
                    dp *= z[j][v] * sig;
                    z[j][v] = g[j][v] * pv * dsilu(z[j][v], sig);
                } else if (p.act == MI_ACT_SILU) {
                    dp *= dsilu(pv, sigmoid(pv));
                }
                if (ok) {  // rows that do not exist have zeros for x and dy, and rstd of nothing
                    dw[j][v] = fmaf(dp, x[j][v], dw[j][v]);
                    db[j][v] += dp;
                }
                g[j][v] = dp * w[j][v];
                c[0] = fmaf(g[j][v], x[j][v], c[0]);
                c[1] += g[j][v];
            }
        team_sum<TEAM>(c, sm);
        const float c1 = c[0] * p.inv_dg, c2 = p.centered ? c[1] * p.inv_dg : 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float f[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) f[v] = rstd * (g[j][v] - c2 - x[j][v] * c1);
            if (ok && H::at(o.q, j) < p.dg) {
                store_vec<T, VEC>(static_cast<T *>(p.dx) + base + H::at(o.q, j), Pack<T, VEC>::pack(f));
                if (p.z) store_vec<T, VEC>(static_cast<T *>(p.dz) + base + H::at(o.q, j), Pack<T, VEC>::pack(z[j]));
            }
        }
    }
    // one partial row of dw and dbias a workgroup
    float *pw = p.part + (int64_t)part * 2 * p.D + o.c0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const int e = H::at(o.q, j) + v;
            if constexpr (TEAM == 256) {
                if (e < p.dg) {
                    pw[e] = dw[j][v];
                    pw[p.D + e] = db[j][v];
                }
            } else {
                __syncthreads();
                acc[0][wave][lane] = dw[j][v];
                acc[1][wave][lane] = db[j][v];
                __syncthreads();
                const int span = TEAM * p.gps;  // lanes of one row
                if (threadIdx.x < 2 * span) {
                    const int k = threadIdx.x / span, l = threadIdx.x % span;
                    float s = 0.f;
                    for (int q = l; q < 64; q += span)
                        s += (acc[k][0][q] + acc[k][1][q]) + (acc[k][2][q] + acc[k][3][q]);
                    const int grp = slice * p.gps + l / TEAM, el = H::at(l % TEAM, j) + v;
                    if (grp < p.G && el < p.dg)
                        p.part[((int64_t)part * 2 + k) * p.D + (int64_t)grp * p.dg + el] = s;
                }
            }
        }
}

// Groups too wide for registers: a workgroup a group and row, the row read
// three times (from the L2 after the first).
template <typename T, bool BWD>
__global__ __launch_bounds__(256) void norm_wide_kernel(NormArgs p) {
    __shared__ float sm[2][4];
    const int g = blockIdx.x % p.G, part = blockIdx.x / p.G;
    const int64_t c0 = (int64_t)g * p.dg;
    const int64_t r0 = (int64_t)part * p.rows;
    const int64_t last = r0 + p.rows < p.R ? r0 + p.rows : p.R;
    float *pw = BWD ? p.part + (int64_t)part * 2 * p.D + c0 : nullptr;
    for (int64_t r = r0; r < last; ++r) {
        const int64_t base = r * p.D + c0;
        const T *x = static_cast<const T *>(p.x) + base;
        const T *z = p.z ? static_cast<const T *>(p.z) + base : nullptr;
        float s[1] = {0.f}, mean = 0.f;
        if (p.centered) {
            for (int e = threadIdx.x; e < p.dg; e += 256) s[0] += ld1(x + e);
            team_sum<256>(s, sm);
            mean = s[0] * p.inv_dg;
        }
        s[0] = 0.f;
        for (int e = threadIdx.x; e < p.dg; e += 256) {
            const float c = ld1(x + e) - mean;
            s[0] = fmaf(c, c, s[0]);
        }
        team_sum<256>(s, sm);
        const float rstd = __builtin_amdgcn_rsqf(fmaf(s[0], p.inv_dg, p.eps));
        if constexpr (!BWD) {
            T *y = static_cast<T *>(p.y) + base;
            for (int e = threadIdx.x; e < p.dg; e += 256) {
                float f = fmaf((ld1(x + e) - mean) * rstd, p.w ? p.w[c0 + e] : 1.f, p.bias ? p.bias[c0 + e] : 0.f);
                if (p.act == MI_ACT_SILU) f = silu(f);
                if (z) f *= silu(ld1(z + e));
                st1(y + e, f);
            }
        } else {
            const T *dy = static_cast<const T *>(p.dy) + base;
            T *dx = static_cast<T *>(p.dx) + base;
            T *dz = p.z ? static_cast<T *>(p.dz) + base : nullptr;
            float c[2] = {0.f, 0.f};
            for (int e = threadIdx.x; e < p.dg; e += 256) {
                const float xh = (ld1(x + e) - mean) * rstd, w = p.w ? p.w[c0 + e] : 1.f;
                const float pv = fmaf(xh, w, p.bias ? p.bias[c0 + e] : 0.f), gy = ld1(dy + e);
                float dp = gy;
                if (z) {
                    const float zz = ld1(z + e), sig = sigmoid(zz);
                    dp *= zz * sig;
                    st1(dz + e, gy * pv * dsilu(zz, sig));
                } else if (p.act == MI_ACT_SILU) {
                    dp *= dsilu(pv, sigmoid(pv));
                }
                pw[e] = r == r0 ? dp * xh : fmaf(dp, xh, pw[e]);
                pw[p.D + e] = r == r0 ? dp : pw[p.D + e] + dp;
                c[0] = fmaf(dp * w, xh, c[0]);
                c[1] = fmaf(dp, w, c[1]);
            }
            team_sum<256>(c, sm);
            const float c1 = c[0] * p.inv_dg, c2 = p.centered ? c[1] * p.inv_dg : 0.f;
            for (int e = threadIdx.x; e < p.dg; e += 256) {
                const float xh = (ld1(x + e) - mean) * rstd, w = p.w ? p.w[c0 + e] : 1.f;
                float dp = ld1(dy + e);
                if (z) dp *= silu(ld1(z + e));
                else if (p.act == MI_ACT_SILU) {
                    const float pv = fmaf(xh, w, p.bias ? p.bias[c0 + e] : 0.f);
                    dp *= dsilu(pv, sigmoid(pv));
                }
                st1(dx + e, rstd * (dp * w - c2 - xh * c1));
            }
        }
    }
}

struct StoreNorm {
    float *dw, *db;
    int64_t D;
    __device__ __forceinline__ void operator()(int64_t m, float s) const {
        if (m < D) {
            if (dw) dw[m] = s;
        } else if (db) {
            db[m - D] = s;
        }
    }
};

// How a shape is cut: lanes a group (1, 4, 16, 64, 256) and vectors a lane, the
// smallest that hold a group: up to 8, and 16 of one or two elements in the backward;
// 0 vectors: the wide kernel.  16384 rows bf16 with a gate, forward and backward: 4096
// channels in 512 groups, one vector each, 233 us with one lane a group and 466 with four.
// 16 elements a lane against the wide kernel, 4096 gated rows of one group, us:
//              forward                                 backward
//   channels   3001       4095      6002      8190      3001       4095       6002       8190
//   bf16       49 / 37    64 / 47   155 / 71  177 / 94  120 / 215  148 / 282  208 / 448  235 / 716
//   fp32       200 / 42   240 / 55  312 / 112 400 / 157 247 / 227  286 / 383  510 / 582  577 / 787
// The wide forward reads a row again from the L2 and keeps more waves; the wide backward
// adds up its gradients in memory.  8 vectors of 16 bytes: bf16 162 / 254 and 421 / 1471
// (16384 channels), fp32 128 / 156 and 226 / 773 (8192).
struct NormPlan {
    int team, nv;
    int64_t slices, parts, rows;
};
NormPlan norm_plan(int64_t R, int64_t D, int64_t G, int vec, bool bwd) {
    NormPlan q;
    const int64_t dg = D / G, n = (dg + vec - 1) / vec;
    q.team = n <= 1 ? 1 : n <= 4 ? 4 : n <= 16 ? 16 : n <= 64 ? 64 : 256;
    q.nv = 1;
    while (q.nv < (vec <= 2 && bwd ? 16 : 8) && (int64_t)q.team * q.nv < n) q.nv *= 2;
    if ((int64_t)q.team * q.nv < n) q.nv = 0;
    int gps = 1;
    if (q.team < 64)
        while (gps < 64 / q.team && gps < G) gps *= 2;
    q.slices = q.team == 256 ? G : (G + gps - 1) / gps;
    // about 2048 workgroups (8 a CU); the backward at most 512 partial rows, which the
    // closing sum reads.  16384 rows bf16, gated, us with 1024 / 2048 / 4096 workgroups
    // forward: 4096 channels in 32 groups 72 / 74 / 65, in one 71 / 71 / 71, 1024 in one 36 /
    // 31 / 29; with 256 / 512 / 1024 rows backward (and the sum): 4096 in 32 groups all 156,
    // in one 298 / 182 / 207, 1024 in one 140 / 86 / 72, 64 in one 20 / 22 / 32
    const int64_t unit = q.team == 256 ? 1 : 4 * (64 / q.team / gps);  // rows of one turn
    const int64_t turns = (R + unit - 1) / unit;
    int64_t parts = (2048 + q.slices - 1) / q.slices;
    if (bwd && parts > 512) parts = 512;
    if (parts > turns) parts = turns;
    if (parts < 1) parts = 1;
    q.rows = (turns + parts - 1) / parts * unit;
    if (q.rows < 1) q.rows = 1;
    q.parts = (R + q.rows - 1) / q.rows;
    return q;
}

int norm_gps(const NormPlan &q, int64_t G) {
    int gps = 1;
    if (q.team < 64)
        while (gps < 64 / q.team && gps < G) gps *= 2;
    return gps;
}

// Vector width: 16 bytes, two elements or one, in whole vectors a group and as the
// pointers are aligned.
int norm_vec(int64_t D, int64_t G, size_t es, const Buf *b, int n) {
    const int maxv = (int)(16 / es), v = pick_vec(D, es, b, n);
    return (D / G) % maxv == 0 && v == maxv ? maxv : (D / G) % 2 == 0 && v >= 2 ? 2 : 1;
}

template <typename T, int VEC, int NV, int TEAM, bool BWD>
mi_status go(const NormArgs &a, unsigned grid, hipStream_t s) {
    if constexpr (BWD) hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, NV, TEAM>), dim3(grid), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, NV, TEAM>), dim3(grid), dim3(256), 0, s, a);
    return launch_status();
}
template <typename T, int VEC, bool BWD>
mi_status launch_norm(const NormArgs &a, const NormPlan &q, unsigned grid, hipStream_t s) {
    if (q.nv == 0) {
        hipLaunchKernelGGL((norm_wide_kernel<T, BWD>), dim3(grid), dim3(256), 0, s, a);
        return launch_status();
    }
    if (q.team == 1) return go<T, VEC, 1, 1, BWD>(a, grid, s);
    if (q.team == 4) return go<T, VEC, 1, 4, BWD>(a, grid, s);
    if (q.team == 16) return go<T, VEC, 1, 16, BWD>(a, grid, s);
    if (q.team == 64) return go<T, VEC, 1, 64, BWD>(a, grid, s);
    switch (q.nv) {
        case 1: return go<T, VEC, 1, 256, BWD>(a, grid, s);
        case 2: return go<T, VEC, 2, 256, BWD>(a, grid, s);
        case 4: return go<T, VEC, 4, 256, BWD>(a, grid, s);
    }
    if constexpr (VEC <= 2 && BWD)
        if (q.nv == 16) return go<T, VEC, 16, 256, BWD>(a, grid, s);
    return go<T, VEC, 8, 256, BWD>(a, grid, s);
}
template <typename T, bool BWD>
mi_status run_norm(NormArgs a, int vec, hipStream_t s, int64_t *parts) {
    const NormPlan q = norm_plan(a.R, a.D, a.G, vec, BWD);
    int64_t grid;
    if (!mul_ok(q.slices, q.parts, 1, 1, &grid) || !launch_fits(grid, 256)) return MI_ERR_UNSUPPORTED;
    a.rows = q.rows;
    a.gps = norm_gps(q, a.G);
    a.n_slices = (int)q.slices;
    *parts = q.parts;
    if (grid == 0) return MI_OK;
    constexpr int V = (int)(16 / sizeof(T));
    if (vec == V) return launch_norm<T, V, BWD>(a, q, (unsigned)grid, s);
    if (vec == 2) return launch_norm<T, 2, BWD>(a, q, (unsigned)grid, s);
    return launch_norm<T, 1, BWD>(a, q, (unsigned)grid, s);
}
template <bool BWD>
mi_status run_norm(const NormArgs &a, mi_dtype dt, int vec, hipStream_t s, int64_t *parts) {
    if (dt == MI_F32) return run_norm<float, BWD>(a, vec, s, parts);
    if (dt == MI_BF16) return run_norm<bf16_t, BWD>(a, vec, s, parts);
    return run_norm<f16_t, BWD>(a, vec, s, parts);
}

mi_status check_norm(int64_t R, int64_t D, int64_t G, float eps, mi_act act, const void *z, mi_dtype dt,
                     int64_t *bytes) {
    if (R < 0 || D < 0 || G < 1 || !(eps >= 0.f)) return MI_ERR_INVALID_ARG;
    if (!dtype_known(dt) || (act != MI_ACT_NONE && act != MI_ACT_SILU)) return MI_ERR_UNSUPPORTED;
    if (D % G != 0 || (z != nullptr && act != MI_ACT_NONE)) return MI_ERR_INVALID_ARG;
    if (G > 0x40000000 || D / G > 0x40000000) return MI_ERR_UNSUPPORTED;
    if (!mul_ok(R, D, (int64_t)elem_size(dt), 1, bytes)) return MI_ERR_INVALID_ARG;
    return MI_OK;
}

}  // namespace
}  // namespace miscan

using namespace miscan;

extern "C" {

mi_status mi_group_norm_fwd(const void *x, const float *w, const float *bias, const void *z, void *y, int64_t R,
                            int64_t D, int64_t G, float eps, int centered, mi_act act, mi_dtype dt,
                            hipStream_t stream) {
    int64_t bytes, parts;
    mi_status st = check_norm(R, D, G, eps, act, z, dt, &bytes);
    if (st != MI_OK || R == 0 || D == 0) return st;
    const size_t es = elem_size(dt);
    BufList in, out;
    in.need(x, bytes, es).opt(w, D * 4, 4).opt(bias, D * 4, 4).opt(z, bytes, es);
    out.need(y, bytes, es);
    if ((st = check_lists(in, out)) != MI_OK) return st;
    const Buf b[3] = {{x, bytes}, {z, bytes}, {y, bytes}};
    NormArgs a{};
    a.x = x; a.z = z; a.w = w; a.bias = bias; a.y = y; a.R = R; a.D = D; a.G = (int)G; a.dg = (int)(D / G);
    a.eps = eps; a.inv_dg = 1.f / (float)(D / G); a.centered = centered != 0; a.act = act;
    return run_norm<false>(a, dt, norm_vec(D, G, es, b, 3), stream, &parts);
}

size_t mi_group_norm_bwd_workspace(int64_t R, int64_t D, int64_t G, mi_dtype dt) {
    int64_t bytes;
    if (check_norm(R, D, G, 0.f, MI_ACT_NONE, nullptr, dt, &bytes) != MI_OK || R == 0 || D == 0) return 0;
    int64_t need = 0;
    for (int vec : {1, 2, (int)(16 / elem_size(dt))}) {  // pointers decide the width: the largest need
        const NormPlan q = norm_plan(R, D, G, vec, true);
        int64_t n;
        if (!mul_ok(q.parts, D, 8, 1, &n)) return 0;
        if (n > need) need = n;
    }
    return (size_t)need;
}

mi_status mi_group_norm_bwd(const void *x, const float *w, const float *bias, const void *z, const void *dy, void *dx,
                            float *dw, float *dbias, void *dz, int64_t R, int64_t D, int64_t G, float eps,
                            int centered, mi_act act, mi_dtype dt, void *ws, size_t ws_bytes, hipStream_t stream) {
    int64_t bytes, parts = 0;
    mi_status st = check_norm(R, D, G, eps, act, z, dt, &bytes);
    if (st != MI_OK) return st;
    if ((w == nullptr) != (dw == nullptr) || (bias == nullptr) != (dbias == nullptr) ||
        (z == nullptr) != (dz == nullptr))
        return MI_ERR_INVALID_ARG;
    if (D == 0) return MI_OK;
    const size_t es = elem_size(dt);
    BufList in, out;
    in.need(x, bytes, es).opt(w, D * 4, 4).opt(bias, D * 4, 4).opt(z, bytes, es).need(dy, bytes, es);
    out.need(dx, bytes, es).opt(dw, D * 4, 4).opt(dbias, D * 4, 4).opt(dz, bytes, es);
    if ((st = check_lists(in, out)) != MI_OK) return st;
    if (R > 0) {
        const size_t need = mi_group_norm_bwd_workspace(R, D, G, dt);
        if (need == 0) return MI_ERR_INVALID_ARG;
        if ((st = check_ws_lists(ws, ws_bytes, need, in, out)) != MI_OK) return st;
        const Buf b[5] = {{x, bytes}, {z, bytes}, {dy, bytes}, {dx, bytes}, {dz, bytes}};
        NormArgs a{};
        a.x = x; a.z = z; a.dy = dy; a.w = w; a.bias = bias; a.dx = dx; a.dz = dz;
        a.part = static_cast<float *>(ws);
        a.R = R; a.D = D; a.G = (int)G; a.dg = (int)(D / G);
        a.eps = eps; a.inv_dg = 1.f / (float)(D / G); a.centered = centered != 0; a.act = act;
        if ((st = run_norm<true>(a, dt, norm_vec(D, G, es, b, 5), stream, &parts)) != MI_OK) return st;
    }
    if (dw == nullptr && dbias == nullptr) return MI_OK;
    return reduce_parts(static_cast<const float *>(ws), parts, 2 * D, StoreNorm{dw, dbias, D}, stream);
}

}  // extern "C"
