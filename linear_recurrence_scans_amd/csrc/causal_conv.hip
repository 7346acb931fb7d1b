// causal_conv.hip -- depthwise causal convolution over time, channels last,
// with an optional SiLU; its gradient; and its single-token step.
//
// The forward streams x once and writes y once: the bound is HBM.  A lane owns
// VEC consecutive channels (8 bytes), a wave R consecutive steps, and the K - 1
// steps before them are read again (they are in the caches: the neighbouring
// wave reads them too).  All of a wave's rows are loaded before the first is
// used, so a wave keeps R + K - 1 rows in flight.  Measured (MI355X, K = 4, SiLU,
// bf16): B = 8, T = 8192, D = 4096 202 us, 5.3 TB/s of x and y (a streaming read and
// write of that size 5.7); with 16 bytes a lane (140 registers for 74) 211 us, with 8, 24
// and 32 steps a wave 218, 206 and 214 us.  Forward and backward at B = 4, T = 4096,
// D = 2048 together 75 us on the GPU; with 16 bytes and 8 steps a batch in the backward
// (115 registers for 98) 87 us.  fp32: B = 4, T = 8192, D = 4096 195 us (5.5 TB/s); forward
// and backward as above 123 us.
//
// Sums over steps (dw, dbias) are fp32: a wave's 16 to 64 steps, four waves, then the
// partial rows.  Their error, 1.2e-7 of the gradient's norm at B = 5, T = 1037, is twice
// what sums in 64 bits leave after one rounding; y and dx are off by 0.7e-7.
#include "block_ops.hpp"
#include "checks.hpp"

namespace miscan {
namespace {

constexpr int CONV_NW = 4;     // waves a workgroup, along time
constexpr int CONV_FWD_R = 16;  // steps a wave

struct ConvArgs {
    const void *x;
    const float *w, *bias;
    const void *x0;
    const int32_t *lengths;
    void *y, *xT;
    const void *dy, *dxT;
    void *dx, *dx0;
    float *part;  // backward: (B * n_tt, K + 1, D) partial sums of dw and dbias
    int64_t T, D;
    int n_dt, n_tt;  // channel tiles, time tiles
    int rows;        // backward: steps a wave
    int act;
};

template <typename T, int VEC>
struct Rows {
    using PK = Pack<T, VEC>;
    using raw_t = typename PK::raw_t;
    const T *x, *x0;  // this sequence's rows at this lane's channels; x0 may be null
    int64_t D, len;
    int K;
    // input row t of the sequence extended to the left by x0 (t >= -(K - 1)); steps
    // at or past the length, and those before the start without x0, are zero
    __device__ __forceinline__ raw_t get(int64_t t, bool lane_ok) const {
        raw_t r = splat<T, VEC>(0.f);
        if (!lane_ok) return r;
        if (t >= 0) {
            if (t < len) r = load_vec<T, VEC>(x + t * D);
        } else if (x0 != nullptr) {
            r = load_vec<T, VEC>(x0 + (t + K - 1) * D);
        }
        return r;
    }
};

template <typename T, int VEC, int K>
__device__ __forceinline__ void load_taps(const float *w, const float *bias, int64_t d, bool ok, float (&wt)[K][VEC],
                                          float (&bs)[VEC]) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        bs[v] = ok && bias != nullptr ? bias[d + v] : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) wt[k][v] = ok ? w[(d + v) * K + k] : 0.f;
    }
}

template <typename T, int VEC, int K>
__global__ __launch_bounds__(CONV_NW * 64) void conv_fwd_kernel(ConvArgs p) {
    using PK = Pack<T, VEC>;
    using raw_t = typename PK::raw_t;
    constexpr int R = CONV_FWD_R;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int item = blockIdx.x;
    const int dt = item % p.n_dt;
    const int tt = item / p.n_dt % p.n_tt;
    const int64_t b = item / p.n_dt / p.n_tt;
    const int64_t d = ((int64_t)dt * 64 + lane) * VEC;
    const bool ok = d < p.D;
    const int64_t len = seq_len(p.lengths, b, p.T);
    const T *x0 = static_cast<const T *>(p.x0);
    const Rows<T, VEC> rows{static_cast<const T *>(p.x) + b * p.T * p.D + d,
                            K > 1 && x0 != nullptr ? x0 + b * (K - 1) * p.D + d : nullptr, p.D, len, K};
    if (K > 1 && tt == 0 && wave == 0 && p.xT != nullptr && ok) {
        T *xT = static_cast<T *>(p.xT) + b * (K - 1) * p.D + d;
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            store_vec<T, VEC>(xT + (int64_t)j * p.D, rows.get(len + j - (K - 1), true));
    }
    const int64_t t0 = ((int64_t)tt * CONV_NW + wave) * R;
    if (t0 >= p.T) return;
    raw_t raw[R + K - 1];
#pragma unroll
    for (int i = 0; i < R + K - 1; ++i) raw[i] = rows.get(t0 + i - (K - 1), ok);
    float wt[K][VEC], bs[VEC];
    load_taps<T, VEC, K>(p.w, p.bias, d, ok, wt, bs);
    if (!ok) return;
    float win[K][VEC];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) PK::unpack(raw[k], win[k]);
    T *y = static_cast<T *>(p.y) + (b * p.T + t0) * p.D + d;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (t0 + r >= p.T) break;
        PK::unpack(raw[r + K - 1], win[(r + K - 1) % K]);
        float acc[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            acc[v] = bs[v];
#pragma unroll
            for (int k = 0; k < K; ++k) acc[v] = fmaf(wt[k][v], win[(r + k) % K][v], acc[v]);
            if (p.act == MI_ACT_SILU) acc[v] = silu(acc[v]);
            if (t0 + r >= len) acc[v] = 0.f;
        }
        store_vec<T, VEC>(y + (int64_t)r * p.D, PK::pack(acc));
    }
}

// Gradient.  A wave walks its steps (and the K - 1 after them, whose ds reach
// back into its dx) once, with windows of K rows of the input and of ds in
// registers: reads x and dy, writes dx, and adds up dw and dbias for its own
// steps.  The workgroup joins its waves' sums in LDS and stores one partial row;
// reduce_parts adds the rows in a fixed order.
template <typename T, int VEC, int K>
__global__ __launch_bounds__(CONV_NW * 64) void conv_bwd_kernel(ConvArgs p) {
    using PK = Pack<T, VEC>;
    using raw_t = typename PK::raw_t;
    constexpr int U = K * ((4 + K - 1) / K);  // steps an iteration: whole turns of the windows
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int item = blockIdx.x;
    const int dt = item % p.n_dt;
    const int tt = item / p.n_dt % p.n_tt;
    const int64_t b = item / p.n_dt / p.n_tt;
    const int64_t d = ((int64_t)dt * 64 + lane) * VEC;
    const bool ok = d < p.D;
    const int64_t len = seq_len(p.lengths, b, p.T);
    const T *x0 = static_cast<const T *>(p.x0);
    const Rows<T, VEC> rows{static_cast<const T *>(p.x) + b * p.T * p.D + d,
                            K > 1 && x0 != nullptr ? x0 + b * (K - 1) * p.D + d : nullptr, p.D, len, K};
    const Rows<T, VEC> dyr{static_cast<const T *>(p.dy) + b * p.T * p.D + d, nullptr, p.D, len, K};
    const int R = p.rows;
    const int64_t t0 = ((int64_t)tt * CONV_NW + wave) * R;
    float wt[K][VEC], bs[VEC], dw[K][VEC], db[VEC];
    load_taps<T, VEC, K>(p.w, p.bias, d, ok, wt, bs);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][v] = 0.f;
    }
    if (t0 < p.T || t0 == 0) {
        float win[K][VEC], dsw[K][VEC];
        // slot (i % K) holds the row of step i; step t0 - (K - 1) + k is in slot k
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) dsw[k][v] = 0.f;
#pragma unroll
        for (int k = 0; k < K - 1; ++k) PK::unpack(rows.get(t0 + k - (K - 1), ok), win[k]);
        T *dx = static_cast<T *>(p.dx) + b * p.T * p.D + d;
        T *dx0 = static_cast<T *>(p.dx0);
        const T *dxT = static_cast<const T *>(p.dxT);
        const int64_t t_end = t0 + R + K - 1;
        for (int64_t tb = t0; tb < t_end; tb += U) {
            raw_t xr[U], gr[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                xr[i] = rows.get(tb + i, ok);
                gr[i] = dyr.get(tb + i, ok);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t t = tb + i;
                const bool own = t < t0 + R && t < len;
                float g[VEC], out[VEC];
                PK::unpack(xr[i], win[(i + K - 1) % K]);
                PK::unpack(gr[i], g);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    float s = bs[v];
#pragma unroll
                    for (int k = 0; k < K; ++k) s = fmaf(wt[k][v], win[(i + k) % K][v], s);
                    float ds = g[v];
                    if (p.act == MI_ACT_SILU) ds *= dsilu(s, sigmoid(s));
                    if (t >= len) ds = 0.f;
                    dsw[(i + K - 1) % K][v] = ds;
                    if (own) {
                        db[v] += ds;
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k][v] = fmaf(ds, win[(i + k) % K][v], dw[k][v]);
                    }
                    out[v] = 0.f;
#pragma unroll
                    for (int k = 0; k < K; ++k) out[v] = fmaf(wt[k][v], dsw[(i + K - 1 - k) % K][v], out[v]);
                }
                const int64_t tau = t - (K - 1);  // the input step whose gradient is complete
                if (ok && tau < t0 + R && (tau >= t0 || t0 == 0)) {
                    if (K > 1 && dxT != nullptr && tau >= len - (K - 1) && tau < len) {
                        float c[VEC];
                        PK::unpack(load_vec<T, VEC>(dxT + (b * (K - 1) + tau - len + K - 1) * p.D + d), c);
#pragma unroll
                        for (int v = 0; v < VEC; ++v) out[v] += c[v];
                    }
                    if (tau >= 0) {
                        if (tau < p.T) {
                            if (tau >= len)
#pragma unroll
                                for (int v = 0; v < VEC; ++v) out[v] = 0.f;
                            store_vec<T, VEC>(dx + tau * p.D, PK::pack(out));
                        }
                    } else if (K > 1 && dx0 != nullptr) {
                        store_vec<T, VEC>(dx0 + (b * (K - 1) + tau + K - 1) * p.D + d, PK::pack(out));
                    }
                }
            }
        }
    }
    __shared__ float sm[CONV_NW][VEC][64];
    float *part = p.part + ((b * p.n_tt + tt) * (K + 1)) * p.D;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) sm[wave][v][lane] = k < K ? dw[k < K ? k : 0][v] : db[v];
        __syncthreads();
        // thread i joins channel i, i + 256, ... of the tile
        for (int c = threadIdx.x; c < 64 * VEC; c += CONV_NW * 64) {
            const int64_t dc = (int64_t)dt * 64 * VEC + c;
            const int l = c / VEC, v = c % VEC;
            if (dc < p.D) part[(int64_t)k * p.D + dc] = (sm[0][v][l] + sm[1][v][l]) + (sm[2][v][l] + sm[3][v][l]);
        }
        __syncthreads();
    }
}

struct StoreTaps {
    float *dw, *db;
    int64_t D, K;
    __device__ __forceinline__ void operator()(int64_t m, float s) const {
        const int64_t k = m / D, d = m - k * D;
        if (k < K) dw[d * K + k] = s;
        else if (db != nullptr) db[d] = s;
    }
};

// One step: the state is read, shifted and written, a thread a vector of channels.
template <typename T, int VEC, int K>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs p, int64_t n) {
    using PK = Pack<T, VEC>;
    using raw_t = typename PK::raw_t;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t nd = p.D / VEC;
    const int64_t b = i / nd, d = (i - b * nd) * VEC;
    raw_t raw[K];
    const T *x0 = static_cast<const T *>(p.x0) + b * (K - 1) * p.D + d;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) raw[k] = load_vec<T, VEC>(x0 + (int64_t)k * p.D);
    raw[K - 1] = load_vec<T, VEC>(static_cast<const T *>(p.x) + b * p.D + d);
    float wt[K][VEC], acc[VEC];
    load_taps<T, VEC, K>(p.w, p.bias, d, true, wt, acc);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float f[VEC];
        PK::unpack(raw[k], f);
#pragma unroll
        for (int v = 0; v < VEC; ++v) acc[v] = fmaf(wt[k][v], f[v], acc[v]);
    }
    if (p.act == MI_ACT_SILU)
#pragma unroll
        for (int v = 0; v < VEC; ++v) acc[v] = silu(acc[v]);
    T *xo = static_cast<T *>(p.xT) + b * (K - 1) * p.D + d;
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
        *reinterpret_cast<raw_t *>(xo + (int64_t)k * p.D) = raw[k + 1];
    *reinterpret_cast<raw_t *>(static_cast<T *>(p.y) + b * p.D + d) = PK::pack(acc);
}

// Calls f(type tag, K constant) for the runtime dtype and K.
template <typename T> struct Tag { using type = T; };
template <int K> struct Num { static constexpr int value = K; };

template <typename T, class F>
mi_status with_k(int64_t K, F f) {
    switch (K) {
        case 1: return f(Tag<T>(), Num<1>());
        case 2: return f(Tag<T>(), Num<2>());
        case 3: return f(Tag<T>(), Num<3>());
        case 4: return f(Tag<T>(), Num<4>());
        case 5: return f(Tag<T>(), Num<5>());
        case 6: return f(Tag<T>(), Num<6>());
        case 7: return f(Tag<T>(), Num<7>());
        case 8: return f(Tag<T>(), Num<8>());
    }
    return MI_ERR_UNSUPPORTED;
}
template <class F>
mi_status with_type(mi_dtype dt, int64_t K, F f) {
    if (dt == MI_F32) return with_k<float>(K, f);
    if (dt == MI_BF16) return with_k<bf16_t>(K, f);
    return with_k<f16_t>(K, f);
}

// Steps a wave of the backward walks.  Every wave repeats K - 1 steps, so long
// runs waste less; short runs give more waves.  The longest run of 16, 32, 64
// that still makes 4096 waves (16 a CU).  K = 4, bf16, us with 16 / 32 / 64 steps (waves
// at 64): B = 8, T = 8192, D = 4096 (16384) 399 / 353 / 344; B = 4, T = 4096, D = 2048
// (2048) 56 / 48 / 56; B = 2, T = 2048, D = 1024 (256) 20 / 28 / 46; few channels, B = 8,
// T = 8192, D = 64 (1024), where 32 would be better: 47 / 41 / 52.
int bwd_rows(int64_t B, int64_t T, int64_t D, int64_t esize) {
    const int64_t tile = 64 * (8 / esize);
    int r = 64;
    while (r > 16 && B * ((D + tile - 1) / tile) * ((T + r - 1) / r) < 4096) r /= 2;
    return r;
}

// Vector width: 8 bytes (wider ones cost the windows' registers), two elements or
// one.  Forward and backward at B = 4, T = 4096, bf16: D = 4094 178 us in pairs and
// 385 in single elements; D = 4092 146 in 8 bytes; D = 4095 389.
int conv_vec(int64_t D, size_t es, const Buf *b, int n) {
    const int v = pick_vec(D, es, b, n), half = (int)(8 / es);
    return v >= half ? half : v >= 2 ? 2 : 1;
}

int64_t time_tiles(int64_t T, int64_t rows) {
    const int64_t n = (T + rows - 1) / rows;
    return n < 1 ? 1 : n;  // an empty sequence still writes its state
}

struct ConvSizes {
    int64_t x, taps, bias, state;  // bytes
};

mi_status check_conv(int64_t B, int64_t T, int64_t D, int64_t K, mi_act act, mi_dtype dt, ConvSizes *s) {
    if (B < 0 || T < 0 || D < 0 || K < 0) return MI_ERR_INVALID_ARG;
    if (!dtype_known(dt) || K < 1 || K > 8) return MI_ERR_UNSUPPORTED;
    if (act != MI_ACT_NONE && act != MI_ACT_SILU) return MI_ERR_UNSUPPORTED;
    const int64_t es = (int64_t)elem_size(dt);
    if (!mul_ok(B, T, D, es, &s->x) || !mul_ok(B, K - 1, D, es, &s->state) || !mul_ok(D, K, 4, 1, &s->taps))
        return MI_ERR_INVALID_ARG;
    s->bias = D * 4;
    return MI_OK;
}

}  // namespace
}  // namespace miscan

using namespace miscan;

extern "C" {

mi_status mi_causal_conv_fwd(const void *x, const float *w, const float *bias, const void *x0, const int32_t *lengths,
                             void *y, void *xT, int64_t B, int64_t T, int64_t D, int64_t K, mi_act act, mi_dtype dt,
                             hipStream_t stream) {
    ConvSizes s;
    mi_status st = check_conv(B, T, D, K, act, dt, &s);
    if (st != MI_OK) return st;
    if (B == 0 || D == 0 || (T == 0 && (K == 1 || xT == nullptr))) return MI_OK;
    const size_t es = elem_size(dt);
    BufList in, out;
    in.need(w, s.taps, 4).opt(bias, s.bias, 4).opt(lengths, B * 4, 4);
    if (T > 0) in.need(x, s.x, es);
    if (K > 1) in.opt(x0, s.state, es);
    if (T > 0) out.need(y, s.x, es);
    if (K > 1) out.opt(xT, s.state, es);
    if ((st = check_lists(in, out)) != MI_OK) return st;
    const Buf act_bufs[4] = {{x, s.x}, {K > 1 ? x0 : nullptr, s.state}, {y, s.x}, {K > 1 ? xT : nullptr, s.state}};
    const int vec = conv_vec(D, es, act_bufs, 4);
    ConvArgs a{};
    a.x = x; a.w = w; a.bias = bias; a.x0 = x0; a.lengths = lengths; a.y = y; a.xT = xT;
    a.T = T; a.D = D; a.act = act;
    const int64_t tile = 64 * vec;
    const int64_t n_dt = (D + tile - 1) / tile, n_tt = time_tiles(T, CONV_NW * CONV_FWD_R);
    int64_t grid;
    if (!mul_ok(B, n_dt, n_tt, 1, &grid) || !launch_fits(grid, CONV_NW * 64)) return MI_ERR_UNSUPPORTED;
    a.n_dt = (int)n_dt; a.n_tt = (int)n_tt;
    return with_type(dt, K, [&](auto tag, auto num) {
        using T_ = typename decltype(tag)::type;
        constexpr int K_ = decltype(num)::value, V = (int)(8 / sizeof(T_));
        if (vec == V)
            hipLaunchKernelGGL((conv_fwd_kernel<T_, V, K_>), dim3((unsigned)grid), dim3(CONV_NW * 64), 0, stream, a);
        else if (vec == 2)
            hipLaunchKernelGGL((conv_fwd_kernel<T_, 2, K_>), dim3((unsigned)grid), dim3(CONV_NW * 64), 0, stream, a);
        else
            hipLaunchKernelGGL((conv_fwd_kernel<T_, 1, K_>), dim3((unsigned)grid), dim3(CONV_NW * 64), 0, stream, a);
        return launch_status();
    });
}

size_t mi_causal_conv_bwd_workspace(int64_t B, int64_t T, int64_t D, int64_t K, mi_dtype dt) {
    ConvSizes s;
    if (check_conv(B, T, D, K, MI_ACT_NONE, dt, &s) != MI_OK || B == 0 || D == 0) return 0;
    const int64_t n_tt = time_tiles(T, (int64_t)CONV_NW * bwd_rows(B, T, D, (int64_t)elem_size(dt)));
    int64_t bytes;
    if (!mul_ok(B, n_tt, (K + 1) * 4, D, &bytes)) return 0;
    return (size_t)bytes;
}

mi_status mi_causal_conv_bwd(const void *x, const float *w, const float *bias, const void *x0, const int32_t *lengths,
                             const void *dy, const void *dxT, void *dx, float *dw, float *dbias, void *dx0, int64_t B,
                             int64_t T, int64_t D, int64_t K, mi_act act, mi_dtype dt, void *ws, size_t ws_bytes,
                             hipStream_t stream) {
    ConvSizes s;
    mi_status st = check_conv(B, T, D, K, act, dt, &s);
    if (st != MI_OK) return st;
    if (D == 0) return MI_OK;
    const size_t es = elem_size(dt);
    BufList in, out;
    in.need(w, s.taps, 4).opt(bias, s.bias, 4);
    out.need(dw, s.taps, 4).opt(dbias, s.bias, 4);
    if (B > 0) {
        in.opt(lengths, B * 4, 4);
        if (T > 0) in.need(x, s.x, es).need(dy, s.x, es);
        if (K > 1) in.opt(x0, s.state, es).opt(dxT, s.state, es);
        if (T > 0) out.need(dx, s.x, es);
        if (K > 1) out.opt(dx0, s.state, es);
    }
    if ((st = check_lists(in, out)) != MI_OK) return st;
    const size_t need = mi_causal_conv_bwd_workspace(B, T, D, K, dt);
    if (B > 0) {
        if (need == 0) return MI_ERR_UNSUPPORTED;
        if ((st = check_ws_lists(ws, ws_bytes, need, in, out)) != MI_OK) return st;
    }
    ConvArgs a{};
    a.x = x; a.w = w; a.bias = bias; a.x0 = x0; a.lengths = lengths; a.dy = dy; a.dxT = dxT; a.dx = dx; a.dx0 = dx0;
    a.part = static_cast<float *>(ws);
    a.T = T; a.D = D; a.act = act;
    a.rows = bwd_rows(B, T, D, (int64_t)es);
    const int64_t n_tt = time_tiles(T, (int64_t)CONV_NW * a.rows);
    if (B > 0) {
        const bool state = K > 1;
        const Buf act_bufs[6] = {{x, s.x},   {dy, s.x}, {dx, s.x}, {state ? x0 : nullptr, s.state},
                                 {state ? dxT : nullptr, s.state}, {state ? dx0 : nullptr, s.state}};
        const int vec = conv_vec(D, es, act_bufs, 6);
        const int64_t tile = 64 * vec;
        const int64_t n_dt = (D + tile - 1) / tile;
        int64_t grid;
        if (!mul_ok(B, n_dt, n_tt, 1, &grid) || !launch_fits(grid, CONV_NW * 64)) return MI_ERR_UNSUPPORTED;
        a.n_dt = (int)n_dt; a.n_tt = (int)n_tt;
        st = with_type(dt, K, [&](auto tag, auto num) {
            using T_ = typename decltype(tag)::type;
            constexpr int K_ = decltype(num)::value, V = (int)(8 / sizeof(T_));
            if (vec == V)
                hipLaunchKernelGGL((conv_bwd_kernel<T_, V, K_>), dim3((unsigned)grid), dim3(CONV_NW * 64), 0, stream, a);
            else if (vec == 2)
                hipLaunchKernelGGL((conv_bwd_kernel<T_, 2, K_>), dim3((unsigned)grid), dim3(CONV_NW * 64), 0, stream, a);
            else
                hipLaunchKernelGGL((conv_bwd_kernel<T_, 1, K_>), dim3((unsigned)grid), dim3(CONV_NW * 64), 0, stream, a);
            return launch_status();
        });
        if (st != MI_OK) return st;
    }
    return reduce_parts(a.part, B * n_tt, (K + 1) * D, StoreTaps{dw, dbias, D, K}, stream);
}

mi_status mi_causal_conv_step(const void *x, const float *w, const float *bias, const void *x0, void *y, void *x_out,
                              int64_t B, int64_t D, int64_t K, mi_act act, mi_dtype dt, hipStream_t stream) {
    ConvSizes s;
    mi_status st = check_conv(B, 1, D, K, act, dt, &s);
    if (st != MI_OK || B == 0 || D == 0) return st;
    const size_t es = elem_size(dt);
    BufList in, out;
    in.need(x, s.x, es).need(w, s.taps, 4).opt(bias, s.bias, 4);
    out.need(y, s.x, es);
    if (K > 1) {
        if (x_out != x0) in.need(x0, s.state, es);  // in place: the state is checked as an output
        out.need(x_out, s.state, es);
    }
    if ((st = check_lists(in, out)) != MI_OK) return st;
    const Buf act_bufs[4] = {{x, s.x}, {y, s.x}, {K > 1 ? x0 : nullptr, s.state}, {K > 1 ? x_out : nullptr, s.state}};
    const int vec = conv_vec(D, es, act_bufs, 4);
    ConvArgs a{};
    a.x = x; a.w = w; a.bias = bias; a.x0 = x0; a.y = y; a.xT = x_out; a.T = 1; a.D = D; a.act = act;
    const int64_t n = B * D / vec;
    const int64_t grid = (n + 255) / 256;
    if (!launch_fits(grid, 256)) return MI_ERR_UNSUPPORTED;
    return with_type(dt, K, [&](auto tag, auto num) {
        using T_ = typename decltype(tag)::type;
        constexpr int K_ = decltype(num)::value, V = (int)(8 / sizeof(T_));
        if (vec == V)
            hipLaunchKernelGGL((conv_step_kernel<T_, V, K_>), dim3((unsigned)grid), dim3(256), 0, stream, a, n);
        else if (vec == 2)
            hipLaunchKernelGGL((conv_step_kernel<T_, 2, K_>), dim3((unsigned)grid), dim3(256), 0, stream, a, n);
        else
            hipLaunchKernelGGL((conv_step_kernel<T_, 1, K_>), dim3((unsigned)grid), dim3(256), 0, stream, a, n);
        return launch_status();
    });
}

}  // extern "C"
