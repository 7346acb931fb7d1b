/*
 * miscan.h -- C ABI of libmiscan.so: parallel prefix scans of the first-order
 * affine recurrence h_t = a_t * h_{t-1} + b_t and its k x k matrix form, as
 * hand-written HIP kernels for gfx950 (MI355X, CDNA4), one GPU.
 *
 * The operations are those of the minGRU documentation page "Triton kernels"
 * (API reference of mingru.triton_scans), section "Kernel entry points":
 * linear_scan_fwd/bwd, parallel_scan_log_fwd and affine_scan_fwd/bwd.  Each
 * entry point below names the entry it implements.
 *
 * Common contract
 * ---------------
 *  - Tensors are device pointers to contiguous row-major storage.  Time is the
 *    second axis: (B, T, D) for the channel scans, (B, T, n, r, c) for the k x k
 *    scan.  Step t = 1..T of the recurrence is row t-1.
 *  - Outputs have the shape and dtype of the corresponding input.  With bf16
 *    or fp16 storage all arithmetic is fp32; results are rounded to the
 *    storage type (nearest-even) once, on store.  Every output element is
 *    written.
 *  - Ownership: the caller allocates every input, output and the workspace.  The
 *    library keeps no device memory and no state between calls, and never
 *    synchronises: a call enqueues its kernels on `stream` and returns.
 *  - Workspace: at least the bytes reported by the matching *_workspace query,
 *    256-byte aligned, contents need not be initialised (the call clears what
 *    it uses, on `stream`, before its scan kernel).  One workspace must not be
 *    used by two calls that may run concurrently (e.g. on two streams).  Word 1
 *    (bytes 4..7) counts cross-workgroup waits that hit their spin limit during
 *    the last call; it is 0 after every correct run.
 *  - Errors: every check runs before anything is enqueued; on any status other
 *    than MI_OK nothing was launched, except MI_ERR_LAUNCH, which reports that
 *    the HIP runtime refused a launch.  A problem with a zero-sized axis returns
 *    MI_OK without launching.  Inputs and outputs must not overlap.  There is no
 *    fallback to any other implementation.
 *  - Sizes are int64.  Element pointers must be aligned to their element size;
 *    wider alignment (16 bytes) and D (or k, v) divisible by the vector width
 *    select the vectorised kernels, other layouts run narrower ones.
 */
#ifndef MISCAN_H
#define MISCAN_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MI_OK = 0,
    MI_ERR_INVALID_ARG = 1, /* null pointer, negative size, byte-size overflow,
                               misaligned element pointer, overlapping buffers */
    MI_ERR_UNSUPPORTED = 2, /* outside the envelope: k not in [1,16], v not in
                               [1,128], a limit that a block operator states
                               below, or a dtype not built for the op */
    MI_ERR_WORKSPACE = 3,   /* workspace NULL or smaller than the query says */
    MI_ERR_LAUNCH = 4,      /* the HIP runtime reported an error at launch */
    MI_ERR_DEVICE = 5,      /* no usable gfx950 device */
    MI_ERR_CAPACITY = 6     /* the problem needs more than the fixed scratch of
                               mi_linear_scan_fwd_noalloc */
} mi_status;

typedef enum {
    MI_F32 = 0,  /* IEEE binary32 storage */
    MI_BF16 = 1, /* bfloat16 storage, fp32 arithmetic */
    MI_F16 = 2   /* IEEE binary16 storage, fp32 arithmetic */
} mi_dtype;

/* Human-readable name of a status code (static storage, never NULL). */
const char *mi_status_string(mi_status s);

/* Analogue of the page's available() probe ("Triton kernels", Availability and
 * registry): MI_OK if `device` is a gfx950 GPU this library can launch on,
 * otherwise MI_ERR_DEVICE with a reason copied into `reason` (may be NULL). */
mi_status mi_device_check(int device, char *reason, size_t reason_len);

/* ------------------------------------------------------------------------ */
/* k = 1 channel scan ("Triton kernels", Kernel entry points:               */
/* linear_scan_fwd, linear_scan_bwd).  Dtypes: MI_F32, MI_BF16, MI_F16.     */
/* ------------------------------------------------------------------------ */

/* Workspace bytes for mi_linear_scan_fwd / mi_linear_scan_bwd on (B, T, D). */
size_t mi_linear_scan_workspace(int64_t B, int64_t T, int64_t D, mi_dtype dt);

/* linear_scan_fwd: a, b (B,T,D) -> A (running product of a) and Bc (the h_0 = 0
 * solution of h_t = a_t h_{t-1} + b_t), both (B,T,D). */
mi_status mi_linear_scan_fwd(const void *a, const void *b, void *A, void *Bc,
                             int64_t B, int64_t T, int64_t D, mi_dtype dt,
                             void *ws, size_t ws_bytes, hipStream_t stream);

/* linear_scan_bwd: reads the forward input a, the forward outputs A, Bc and the
 * upstream grads gA, gBc (all (B,T,D)); writes da, db (B,T,D), the grads of
 * <gA, A> + <gBc, Bc> with respect to a and b.  A and Bc are used as given:
 * da_t = lam_t Bc_{t-1} + mu_t A_{t-1}, db_t = lam_t, with
 * lam_t = gBc_t + a_{t+1} lam_{t+1}, mu_t = gA_t + a_{t+1} mu_{t+1},
 * a_{T+1} = 0, A_0 = 1, Bc_0 = 0. */
mi_status mi_linear_scan_bwd(const void *a, const void *A, const void *Bc,
                             const void *gA, const void *gBc, void *da, void *db,
                             int64_t B, int64_t T, int64_t D, mi_dtype dt,
                             void *ws, size_t ws_bytes, hipStream_t stream);

/* The same forward as mi_linear_scan_fwd, through an entry point that
 * allocates nothing and takes no workspace.  For callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc.  The look-back workspace is a file-scope device array
 * of MI_NOALLOC_SCRATCH_BYTES inside the library, one per GPU, held until the
 * process ends; the call makes no hipMalloc/hipFree and no allocating library
 * call.  Its device address is looked up (hipGetSymbolAddress) on the first
 * call on each device, which must be the current device and the stream's.
 * The array keeps the last call's contents; each call clears what must start
 * at zero, on `stream`, before its scan kernel.  Every call on one GPU uses
 * the same array: calls that may overlap on one GPU (other streams, other
 * threads) race and must be serialised by the caller.  Same dtypes, layouts,
 * results and argument checks as mi_linear_scan_fwd; a problem whose
 * workspace exceeds the array returns MI_ERR_CAPACITY before anything is
 * enqueued.  72 MiB covers the forward of 2^28 channel-steps in either dtype
 * (e.g. B=8, T=8192, D=4096), about 4.2 bytes of scratch per 16 channel-steps. */
#define MI_NOALLOC_SCRATCH_BYTES (72u << 20)
mi_status mi_linear_scan_fwd_noalloc(const void *a, const void *b, void *A, void *Bc,
                                     int64_t B, int64_t T, int64_t D, mi_dtype dt,
                                     hipStream_t stream);

/* Scans from a given initial state.  The page's linear_scan_fwd returns Bc,
 * the solution from h_0 = 0, and leaves the initial state to the caller
 * (h_t = A_t h_0 + Bc_t).  These two calls take h_0 directly; they are what a
 * caller that carries state across calls (a sequence processed in pieces, or
 * split in time across devices) needs.
 *
 * mi_linear_scan_fwd_h0: h0 (B, D), or NULL for a zero state.  Writes A (the
 * running product, as mi_linear_scan_fwd) and H (B, T, D) with
 * H_t = a_t H_{t-1} + b_t, H_0 = h0.  The final state (A_T, H_T) is the last
 * row of A and H.
 * mi_linear_scan_bwd_h0: the gradient for L = <gA, A> + <gH, H>: da, db as
 * mi_linear_scan_bwd with H in place of Bc and h0 as the state before the
 * first step, and dh0 (B, D) = dL/dh0 = a_1 lam_1 (zero when T = 0).
 * Same dtypes, layouts, workspace (mi_linear_scan_workspace) and errors as the
 * calls above; h0 and dh0 must be aligned like the other tensors and must not
 * overlap outputs. */
mi_status mi_linear_scan_fwd_h0(const void *a, const void *b, const void *h0, void *A, void *H,
                                int64_t B, int64_t T, int64_t D, mi_dtype dt,
                                void *ws, size_t ws_bytes, hipStream_t stream);
mi_status mi_linear_scan_bwd_h0(const void *a, const void *A, const void *H, const void *h0,
                                const void *gA, const void *gH, void *da, void *db, void *dh0,
                                int64_t B, int64_t T, int64_t D, mi_dtype dt,
                                void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Log-space scan ("Triton kernels", Kernel entry points:                   */
/* parallel_scan_log_fwd).  Dtypes: MI_F32, MI_BF16, MI_F16.                */
/* ------------------------------------------------------------------------ */

/* Workspace bytes for mi_scan_log_fwd and mi_scan_log_bwd on (B, T, D). */
size_t mi_scan_log_workspace(int64_t B, int64_t T, int64_t D, mi_dtype dt);

/* parallel_scan_log_fwd: log_coeffs (B,T,D) holds log a_t; log_values (B,T+1,D)
 * holds log h_0 in slot 0 and log b_t in slots 1..T.  Writes h_1..h_T as one
 * (B,T,D) tensor `h`, where h_t = a_t h_{t-1} + b_t.  The scan state is kept in
 * log space (log-sum-exp combine); only the stored states are exponentiated. */
mi_status mi_scan_log_fwd(const void *log_coeffs, const void *log_values, void *h,
                          int64_t B, int64_t T, int64_t D, mi_dtype dt,
                          void *ws, size_t ws_bytes, hipStream_t stream);

/* Gradient of parallel_scan_log_fwd.  The page defines the log-space scan as
 * a forward op; this is the adjoint of that forward definition, for training
 * through it.  Inputs: log_coeffs (B,T,D) and log_values (B,T+1,D) as in the
 * forward, h (B,T,D) the forward output, g (B,T,D) the upstream gradient
 * dL/dh.  Outputs: dlog_coeffs (B,T,D) and dlog_values (B,T+1,D), slot 0 being
 * the gradient of log h_0:
 *     lam_t = g_t + a_{t+1} lam_{t+1} (a_{T+1} = 0),
 *     dlog_coeffs_t = lam_t a_t h_{t-1},  dlog_values_t = lam_t b_t (t >= 1),
 *     dlog_values_0 = a_1 lam_1 h_0,
 * with a = exp(log_coeffs), b and h_0 = exp(log_values), and h_{t-1} taken
 * from the given h (not recomputed).  lam runs in linear space (g is
 * signed).  Outputs must not overlap inputs or each other; all arithmetic is
 * fp32, storage as dt.  With T = 0 (and B, D > 0) the only output is slot 0 of
 * dlog_values, which is set to zero; the other pointers are not used. */
mi_status mi_scan_log_bwd(const void *log_coeffs, const void *log_values, const void *h,
                          const void *g, void *dlog_coeffs, void *dlog_values,
                          int64_t B, int64_t T, int64_t D, mi_dtype dt,
                          void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* k x k matrix-affine scan ("Triton kernels", Kernel entry points:         */
/* affine_scan_fwd, affine_scan_bwd).  Dtypes: MI_F32, MI_BF16, MI_F16     */
/* (storage; arithmetic fp32).  1 <= k <= 16,                               */
/* 1 <= v <= 128.                                                           */
/* ------------------------------------------------------------------------ */

/* Workspace bytes for mi_affine_scan_fwd / mi_affine_scan_bwd. */
size_t mi_affine_scan_workspace(int64_t B, int64_t T, int64_t n, int64_t k,
                                int64_t v, mi_dtype dt);

/* affine_scan_fwd: A (B,T,n,k,k), Bm (B,T,n,k,v) -> Abar (B,T,n,k,k), the
 * running product A_t @ ... @ A_1 (composition A_current @ A_earlier), and Bbar
 * (B,T,n,k,v), the H_0 = 0 solution of H_t = A_t @ H_{t-1} + Bm_t. */
mi_status mi_affine_scan_fwd(const void *A, const void *Bm, void *Abar, void *Bbar,
                             int64_t B, int64_t T, int64_t n, int64_t k, int64_t v,
                             mi_dtype dt, void *ws, size_t ws_bytes,
                             hipStream_t stream);

/* affine_scan_bwd: reads the forward input A, the forward outputs Abar, Bbar and
 * the upstream grads gAbar (shape of Abar), gBbar (shape of Bbar); writes dA
 * (shape of A) and dB (shape of Bbar), the grads of <gAbar, Abar> +
 * <gBbar, Bbar> with respect to A and Bm.  With M_t = gAbar_t + A_{t+1}^T M_{t+1}
 * and Lam_t = gBbar_t + A_{t+1}^T Lam_{t+1} (nothing after T):
 * dB_t = Lam_t, dA_t = M_t Abar_{t-1}^T + Lam_t Bbar_{t-1}^T, Abar_0 = I,
 * Bbar_0 = 0.  Abar and Bbar are used as given. */
mi_status mi_affine_scan_bwd(const void *A, const void *Abar, const void *Bbar,
                             const void *gAbar, const void *gBbar, void *dA, void *dB,
                             int64_t B, int64_t T, int64_t n, int64_t k, int64_t v,
                             mi_dtype dt, void *ws, size_t ws_bytes,
                             hipStream_t stream);

/* Scans from a given initial state (the k x k counterpart of
 * mi_linear_scan_fwd_h0 / _bwd_h0).  The page's affine_scan_fwd returns Bbar,
 * the solution from H_0 = 0.
 * mi_affine_scan_fwd_h0: H0 (B, n, k, v), or NULL for zero.  Writes Abar (as
 * mi_affine_scan_fwd) and H (B,T,n,k,v), H_t = A_t H_{t-1} + Bm_t, H_0 = H0;
 * equivalently X_t = A_t X_{t-1} + [0 | Bm_t] from X_0 = [I | H0].
 * mi_affine_scan_bwd_h0: gradient for L = <gAbar, Abar> + <gH, H>: dA, dB as
 * mi_affine_scan_bwd with H in place of Bbar and H0 as the state before the
 * first step (dA_1 = M_1 + Lam_1 H0^T), and dH0 (B,n,k,v) = A_1^T Lam_1 (zero
 * when T = 0).  Same dtype, envelope, workspace and errors as the calls
 * above; H0 and dH0 must not overlap outputs. */
mi_status mi_affine_scan_fwd_h0(const void *A, const void *Bm, const void *H0, void *Abar, void *H,
                                int64_t B, int64_t T, int64_t n, int64_t k, int64_t v, mi_dtype dt,
                                void *ws, size_t ws_bytes, hipStream_t stream);
mi_status mi_affine_scan_bwd_h0(const void *A, const void *Abar, const void *H, const void *H0,
                                const void *gAbar, const void *gH, void *dA, void *dB, void *dH0,
                                int64_t B, int64_t T, int64_t n, int64_t k, int64_t v, mi_dtype dt,
                                void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Block operators: what a recurrent sequence layer runs around its scan.   */
/*                                                                          */
/* Activations (x, u, delta, z, Bm, Cm and their gradients) have the dtype  */
/* `dt`; parameters (w, bias, A, skip, delta_bias and their gradients) and  */
/* scan states are fp32.  All arithmetic is fp32.  Results are bitwise      */
/* reproducible: sums over rows and channels have a fixed order and no      */
/* floating-point atomics are used.  `lengths` (B int32 on the device, or   */
/* NULL for T each) gives every sequence its own length; values are clamped */
/* to [0, T].  Steps at or past it are not read into any result (they may   */
/* hold anything, NaN included); outputs and gradients there are zero.      */
/*                                                                          */
/* A launch holds fewer than 2^32 threads: a call that needs more, such as  */
/* the scan's backward for 2^23 sequences, is MI_ERR_UNSUPPORTED.           */
/* ------------------------------------------------------------------------ */

typedef enum {
    MI_ACT_NONE = 0,
    MI_ACT_SILU = 1 /* x / (1 + exp(-x)) */
} mi_act;

/* Causal convolution, depthwise, channels last.  x (B,T,D), w (D,K), bias (D)
 * or NULL, x0 (B,K-1,D) the inputs before the first step or NULL for zeros.
 * With xe = [x0 ; x] along time:
 *     s_t = bias + sum_{k<K} w[:,k] xe_{t+k},   y_t = act(s_t),
 * and xT (B,K-1,D), or NULL: the K-1 inputs that end at the sequence's
 * length, the x0 of its continuation (an exact copy).  1 <= K <= 8.
 * With K = 1, x0 and xT hold nothing and are not used. */
mi_status mi_causal_conv_fwd(const void *x, const float *w, const float *bias, const void *x0,
                             const int32_t *lengths, void *y, void *xT, int64_t B, int64_t T,
                             int64_t D, int64_t K, mi_act act, mi_dtype dt, hipStream_t stream);

/* Gradient of the above for the upstream gradients dy (B,T,D) and dxT
 * (B,K-1,D) or NULL: dx (B,T,D), dw (D,K), dbias (D) or NULL, dx0 (B,K-1,D) or
 * NULL.  s is recomputed.  ds = dy act'(s); dx_t = sum_k w[:,k] ds_{t+K-1-k}
 * (+ dxT); dw[:,k] = sum_{b,t} ds_t xe_{t+k}; dbias = sum ds. */
size_t mi_causal_conv_bwd_workspace(int64_t B, int64_t T, int64_t D, int64_t K, mi_dtype dt);
mi_status mi_causal_conv_bwd(const void *x, const float *w, const float *bias, const void *x0,
                             const int32_t *lengths, const void *dy, const void *dxT, void *dx,
                             float *dw, float *dbias, void *dx0, int64_t B, int64_t T, int64_t D,
                             int64_t K, mi_act act, mi_dtype dt, void *ws, size_t ws_bytes,
                             hipStream_t stream);

/* One step of the convolution: x (B,D), x0 (B,K-1,D) -> y (B,D) and x_out
 * (B,K-1,D), x0 shifted by one with x appended.  x_out may be x0 itself
 * (update in place); no other overlap is allowed. */
mi_status mi_causal_conv_step(const void *x, const float *w, const float *bias, const void *x0,
                              void *y, void *x_out, int64_t B, int64_t D, int64_t K, mi_act act,
                              mi_dtype dt, hipStream_t stream);

/* Selective state-space scan: N states a channel, with gates formed from the
 * token.  u, delta, z (B,T,D); A (D,N); Bm, Cm (B,T,G,N), one row for the D/G
 * channels of a group; skip, delta_bias (D); h0, hT (B,D,N).  z, skip,
 * delta_bias, h0, hT may be NULL.  1 <= N <= 64, G divides D, and D and G N
 * are at most 2^24.
 *     dl_t = softplus(delta_t + delta_bias)       (softplus = 0: delta + bias)
 *     h_t[n] = exp(dl_t A[n]) h_{t-1}[n] + dl_t u_t Bm_t[n],   h_0 = h0
 *     s_t = sum_n Cm_t[n] h_t[n] + skip u_t,   y_t = s_t silu(z_t)
 * hT is the state at the sequence's length.  `states`, or NULL, receives what
 * the backward needs: the fp32 state before every block of
 * mi_selective_scan_block(N) steps, (B, ceil(T/block), D, N).  The workspace
 * holds the transforms of a sequence's segments where the channels alone do
 * not fill the GPU; it may be NULL where the query says 0 bytes.
 *
 * Non-finite values.  A result that the formulas make infinite may be NaN
 * instead (steps are composed, and inf 0 arises where one step after the other
 * would keep the infinity); a result that does not depend on a non-finite input
 * is not touched by it.  Rates of growth (exp(dl A) > 1) are finite in the
 * results as long as every gate, state and gradient is.  A may be -inf: such a
 * state keeps its value over steps of rate zero and forgets it over any other. */
int64_t mi_selective_scan_block(int64_t N);
size_t mi_selective_scan_fwd_workspace(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, mi_dtype dt);
mi_status mi_selective_scan_fwd(const void *u, const void *delta, const float *A, const void *Bm,
                                const void *Cm, const float *skip, const void *z,
                                const float *delta_bias, const float *h0, const int32_t *lengths,
                                void *y, float *hT, float *states, int64_t B, int64_t T, int64_t D,
                                int64_t G, int64_t N, int softplus, mi_dtype dt, void *ws,
                                size_t ws_bytes, hipStream_t stream);

/* Gradient for the upstream gradients dy (B,T,D) and dhT (B,D,N) or NULL.
 * `states` is the forward's.  dskip, dz, ddelta_bias go with skip, z and
 * delta_bias (NULL together); dh0 may be NULL.  With ds = dy silu(z),
 * g_t = Cm_t ds_t + a_{t+1} g_{t+1} (g_T includes dhT), q_t = g_t a_t h_{t-1}:
 *     dCm_t = sum_ch ds_t h_t,  dBm_t = sum_ch g_t dl_t u_t,
 *     dA = sum_t q_t dl_t,      ddl_t = sum_n q_t A + u_t sum_n g_t Bm_t,
 *     du_t = dl_t sum_n g_t Bm_t + skip ds_t,   dh0 = a_1 g_1. */
size_t mi_selective_scan_bwd_workspace(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, mi_dtype dt);
mi_status mi_selective_scan_bwd(const void *u, const void *delta, const float *A, const void *Bm,
                                const void *Cm, const float *skip, const void *z,
                                const float *delta_bias, const float *states,
                                const int32_t *lengths, const void *dy, const float *dhT, void *du,
                                void *ddelta, float *dA, void *dBm, void *dCm, float *dskip,
                                void *dz, float *ddelta_bias, float *dh0, int64_t B, int64_t T,
                                int64_t D, int64_t G, int64_t N, int softplus, mi_dtype dt,
                                void *ws, size_t ws_bytes, hipStream_t stream);

/* One step of the scan: u, delta, z (B,D), Bm, Cm (B,G,N), h (B,D,N) -> y (B,D)
 * and h_out (B,D,N), which may be h itself (update in place). */
mi_status mi_selective_scan_step(const void *u, const void *delta, const float *A, const void *Bm,
                                 const void *Cm, const float *h, const float *skip, const void *z,
                                 const float *delta_bias, void *y, float *h_out, int64_t B,
                                 int64_t D, int64_t G, int64_t N, int softplus, mi_dtype dt,
                                 hipStream_t stream);

/* Group norm, channels last: x (R,D), the D/G channels of a group of one row
 * are normalised together (nothing crosses rows, so it is causal in time).
 *     xh = (x - mean) / sqrt(var + eps)             (centered)
 *     xh = x / sqrt(mean(x^2) + eps)                (not centered)
 *     p = xh w + bias,   y = act(p) silu(z)
 * w, bias (D) and z (R,D) may be NULL; act and z exclude each other. */
mi_status mi_group_norm_fwd(const void *x, const float *w, const float *bias, const void *z,
                            void *y, int64_t R, int64_t D, int64_t G, float eps, int centered,
                            mi_act act, mi_dtype dt, hipStream_t stream);

/* Gradient for the upstream gradient dy (R,D): dx (R,D), dw, dbias (D), dz (R,D);
 * dw, dbias and dz go with w, bias and z (NULL together).  The statistics are
 * recomputed from x. */
size_t mi_group_norm_bwd_workspace(int64_t R, int64_t D, int64_t G, mi_dtype dt);
mi_status mi_group_norm_bwd(const void *x, const float *w, const float *bias, const void *z,
                            const void *dy, void *dx, float *dw, float *dbias, void *dz, int64_t R,
                            int64_t D, int64_t G, float eps, int centered, mi_act act, mi_dtype dt,
                            void *ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MISCAN_H */
