/*
 * wkv_b200.h -- C ABI of the B200 (sm_100a) RWKV-4 WKV forward and
 * per-channel diagonal linear scan library (libwkv_b200.so).
 *
 * Operations
 * ----------
 * wkv_forward / wkv_forward_bf16
 *   The RWKV-4 time-mixing WKV operator, eq. (14) of "RWKV：基于RNN的LLM"
 *   (section 二.1, Time-mixing block), written 0-based: for every batch row
 *   b, channel c and step t,
 *
 *     y[b,t,c] = ( sum_{i<t} e^{-(t-1-i) w[c] + k[b,i,c]} v[b,i,c] + e^{u[c] + k[b,t,c]} v[b,t,c] )
 *              / ( sum_{i<t} e^{-(t-1-i) w[c] + k[b,i,c]}          + e^{u[c] + k[b,t,c]} )
 *
 *   w is the per-channel decay, non-negative per eq. (10) of the same page
 *   (section 一.2); u is the bonus of the current token.  y[b,0,c] = v[b,0,c].
 *
 * diag_scan
 *   The per-channel diagonal linear recurrence the LRU and minGRU pages reduce
 *   their RNNs to ("Were RNNs All We Needed?", model-architecture section:
 *   v_t = a_t (.) v_{t-1} + b_t; review of "Resurrecting Recurrent Neural
 *   Networks for Long Sequences", linear-RNN section):
 *
 *     h[b,t,d] = a[b,t,d] * h[b,t-1,d] + b[b,t,d],    h[b,-1,d] = h0[b,d] (or 0).
 *
 * gated_delta, group_norm
 *   The recurrence with a matrix state per head (the gated delta rule) and the
 *   normalisation with an activated gate that follows it; each with gradients.
 *   Their layouts and scratch are described at the declarations.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layout    k, v, y, a, b, h are dense row-major [B, T, C] (or [B, T, D])
 *           tensors with the channel index fastest; w, u are [C]; h0 is [B, D].
 * Memory    every pointer is a DEVICE pointer on the current CUDA device,
 *           owned by the caller.  Outputs must not overlap inputs.
 * Streams   calls are asynchronous on `stream` (NULL = legacy default stream):
 *           a return of WKV_OK means the work was queued.
 * Types     fp32 entry points read and write IEEE float.  wkv_forward_bf16
 *           reads k, v and writes y as bfloat16 bit patterns (wkv_bf16_t),
 *           computes in fp32 and rounds y to nearest even; w, u stay fp32.
 * Sizes     B, T, C (D) >= 0; an empty tensor (any size 0) is a no-op.
 *           B*T*C must be < 2^62.
 * Scratch   inputs with T longer than one tile carry state between thread
 *           blocks through a small library-owned device workspace, one per
 *           (device, stream), allocated with cudaMalloc on first use and
 *           grown when a larger problem needs it.  The tile length is chosen
 *           per call (wkv_tile_steps_for() below returns it; unless
 *           wkv_set_tile_steps() fixed it): 128 steps, or 256 for sequences
 *           longer than 4096 steps with fewer than 64 tiles per time
 *           segment.  Make one call of each size before capturing a stream
 *           into a CUDA graph.  Calls on different streams use different
 *           workspaces and may run concurrently.
 * Rounding  results match the operator to fp32 rounding.  They are bitwise
 *           reproducible from run to run when T spans at most two tiles
 *           (256 steps at the 128-step default, 512 where the call takes
 *           256-step tiles).  Beyond that the carry between tiles may fold
 *           a different, equivalent set of partial results, which can move
 *           the last bits.
 * Errors    argument errors are detected on the host before anything is
 *           launched and return a non-zero wkv_status; wkv_last_error()
 *           then describes the problem (thread-local, valid until the next
 *           call on that thread).  Value preconditions (w >= 0, finite
 *           inputs) are documented, not checked: NaN propagates.
 *           A device-side wait that gives up (see wkv_device_status) writes
 *           NaN outputs for the affected tile and raises WKV_ERR_TIMEOUT
 *           instead of hanging (where a declaration below does not say
 *           otherwise).
 */
#ifndef WKV_B200_H
#define WKV_B200_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define WKV_API __attribute__((visibility("default")))
#else
#define WKV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    WKV_OK = 0,
    WKV_ERR_INVALID_ARG = 1,  /* bad size, NULL pointer, overlapping output  */
    WKV_ERR_ALIGNMENT = 2,    /* pointer not aligned to its element size     */
    WKV_ERR_CUDA = 3,         /* a CUDA runtime/driver call failed           */
    WKV_ERR_TIMEOUT = 4,      /* a bounded device-side wait gave up          */
    WKV_ERR_OOM = 5           /* workspace allocation failed                 */
} wkv_status;

/* bfloat16 storage: the upper 16 bits of the IEEE float32 pattern */
typedef uint16_t wkv_bf16_t;

/* WKV forward, fp32 I/O.  k, v, y: [B, T, C] float; w, u: [C] float.
 * Pointers must be 4-byte aligned.  (16-byte aligned pointers with C a
 * multiple of 4 take the TMA tile path; anything else takes the same kernel
 * with element-wise tile loads.) */
WKV_API wkv_status wkv_forward(int64_t B, int64_t T, int64_t C,
                       const float *w, const float *u,
                       const float *k, const float *v, float *y,
                       cudaStream_t stream);

/* WKV forward, bfloat16 k/v/y with fp32 state.  w, u: [C] float.
 * Pointers must be 2-byte aligned (TMA path: 16-byte and C % 8 == 0). */
WKV_API wkv_status wkv_forward_bf16(int64_t B, int64_t T, int64_t C,
                            const float *w, const float *u,
                            const wkv_bf16_t *k, const wkv_bf16_t *v, wkv_bf16_t *y,
                            cudaStream_t stream);

/* WKV forward from a given state, with the state after the last step
 * returned: streaming a sequence over several calls, and RNN-mode decoding
 * one token per call (T = 1).  The RNN-mode reading of eq. (14) (RWKV
 * evolution article, section RWKV-V4; "RWKV：基于RNN的LLM" section 三,
 * sequential decoding): the state before step t is the pair of past sums
 *
 *     num_t = sum_{i<t} e^{-(t-1-i) w + k_i} v_i,   den_t = the same without v_i,
 *
 * and each step decays it by e^{-w} and adds e^{k_t} (v_t, 1), so a state
 * handed in as the sums before step 0 enters step t weighted by e^{-t w}:
 *
 *     y_t = (e^{-t w} num_in + sum_{0<=i<t} ... + e^{u+k_t} v_t)
 *         / (e^{-t w} den_in + sum_{0<=i<t} ... + e^{u+k_t}).
 *
 * State layout: s_in, s_out are [B, 3, C] float -- for batch row b the planes
 * a, b, p of C floats each, standing for (num, den) = (a, b) * e^p (p in
 * natural-log units; any scaling of one state is the same state).  s_in NULL,
 * or a = b = 0, or p = -inf, is the empty past (then this is wkv_forward).
 * A valid non-empty state has b > 0 and finite fields.  s_out NULL: no state
 * out.  The library writes s_out with b > 0 and p the scale it computed in.
 * Passing the s_out of one call as the s_in of the next continues the
 * sequence (the outputs equal those of one call over all steps, within
 * rounding).  s_out may be the same buffer as s_in (update in place); any
 * other overlap between s_in, s_out and k, v, y, w, u is WKV_ERR_INVALID_ARG.
 * Other arguments, checks and layout as wkv_forward / wkv_forward_bf16;
 * s_in / s_out need 4-byte alignment.  Sequences of at most 16 steps (and
 * wkv_forward's too) run on a kernel that keeps each channel's state in one
 * thread's registers and needs no workspace. */
WKV_API wkv_status wkv_forward_state(int64_t B, int64_t T, int64_t C,
                                     const float *w, const float *u,
                                     const float *k, const float *v, float *y,
                                     const float *s_in, float *s_out,
                                     cudaStream_t stream);

/* wkv_forward_state with bfloat16 k/v/y (fp32 w, u and fp32 state). */
WKV_API wkv_status wkv_forward_bf16_state(int64_t B, int64_t T, int64_t C,
                                          const float *w, const float *u,
                                          const wkv_bf16_t *k, const wkv_bf16_t *v,
                                          wkv_bf16_t *y, const float *s_in, float *s_out,
                                          cudaStream_t stream);

/* WKV forward with the receptance gate fused into its output: eq. (15) of
 * "RWKV：基于RNN的LLM" (section 二.1) applies sigma(r_t) (.) wkv_t before the
 * output projection (the same gate closes the RWKV form in the review of
 * "Resurrecting Recurrent Neural Networks for Long Sequences"), so
 *
 *     y[b,t,c] = wkv[b,t,c] / (1 + e^{-r[b,t,c]})
 *
 * with wkv as in wkv_forward_state.  r: [B, T, C] of the I/O type, read in the
 * same pass as k and v, so the gate costs one extra input stream and no extra
 * output round trip.  s_in / s_out: as wkv_forward_state (either may be NULL).
 * r must not overlap y or s_out; other arguments, checks and layout as
 * wkv_forward_state. */
WKV_API wkv_status wkv_forward_gated(int64_t B, int64_t T, int64_t C,
                                     const float *w, const float *u,
                                     const float *k, const float *v, const float *r, float *y,
                                     const float *s_in, float *s_out, cudaStream_t stream);

/* wkv_forward_gated with bfloat16 k/v/r/y (fp32 w, u and fp32 state). */
WKV_API wkv_status wkv_forward_bf16_gated(int64_t B, int64_t T, int64_t C,
                                          const float *w, const float *u,
                                          const wkv_bf16_t *k, const wkv_bf16_t *v,
                                          const wkv_bf16_t *r, wkv_bf16_t *y,
                                          const float *s_in, float *s_out, cudaStream_t stream);

/* Token shift, the prologue of the time-mixing block: eqs. (11)-(13) of
 * "RWKV：基于RNN的LLM" (section 二.1) feed each projection the interpolation
 *
 *     out[m, b, t, c] = mu[m, c] * x[b, t, c] + (1 - mu[m, c]) * x[b, t-1, c]
 *
 * of every token with the one before it, one mixing vector per projection
 * (the pages also print eqs. (16)-(17) with a minus sign; the plus of eqs.
 * (11)-(13) is the reading taken).  All n_mix (1..4) interpolations come from
 * one read of x.  x[b, -1] is x_prev[b] (the last token of the previous call,
 * the layer's saved "last_x" in the HarmonyOS RWKV article's time-mixing
 * code), or 0 when x_prev is NULL; x_last (if not NULL) receives x[b, T-1].
 * Layout: x [B, T, C]; mu [n_mix, C] float; out [n_mix, B, T, C] (one dense
 * [B, T, C] tensor per mixing vector); x_prev, x_last [B, C].  x_last may be
 * the same buffer as x_prev (update in place); out must not overlap any
 * input, nor x_last.  mu = 1 reproduces x and mu = 0 the shifted x exactly. */
WKV_API wkv_status wkv_token_shift(int64_t B, int64_t T, int64_t C, int64_t n_mix,
                                   const float *x, const float *x_prev, const float *mu,
                                   float *out, float *x_last, cudaStream_t stream);

/* wkv_token_shift on bfloat16 x / x_prev / out / x_last (fp32 mu; computed in
 * fp32, rounded to nearest even). */
WKV_API wkv_status wkv_token_shift_bf16(int64_t B, int64_t T, int64_t C, int64_t n_mix,
                                        const wkv_bf16_t *x, const wkv_bf16_t *x_prev,
                                        const float *mu, wkv_bf16_t *out, wkv_bf16_t *x_last,
                                        cudaStream_t stream);

/* Diagonal linear scan, fp32.  a, b, h: [B, T, D] float; h0: [B, D] float or
 * NULL (zero initial state).  Pointers must be 4-byte aligned. */
WKV_API wkv_status diag_scan(int64_t B, int64_t T, int64_t D,
                     const float *a, const float *b, const float *h0, float *h,
                     cudaStream_t stream);

/* Gradients of the fp32 WKV forward (no state in): given gy = dL/dy [B, T, C],
 * writes gk, gv [B, T, C] and gw, gu [C] (summed over batch rows and steps).
 * The pages give no gradient formulas; eq. (14) of "RWKV：基于RNN的LLM" is a
 * softmax-weighted mean of v_0..v_t with logits l_{t,j} = -(t-1-j) w + k_j
 * (j < t) and l_{t,t} = u + k_t, weights beta_{t,j}, so
 *     gv_j = sum_{t>=j} gy_t beta_{t,j},   gk_j = sum_{t>=j} gy_t beta_{t,j} (v_j - y_t),
 *     gu   = sum_t gy_t beta_{t,t} (v_t - y_t),
 *     gw   = -sum_t sum_{j<t} (t-1-j) gy_t beta_{t,j} (v_j - y_t).
 * Time-parallel over segments of steps, recomputing the forward outputs per
 * segment and running the sums over later outputs backwards in time,
 * max-stabilised (every exponent <= 0 for finite inputs).  When every
 * pointer is 16-byte aligned and C is a multiple of 4 (rows a tensor map
 * can describe): 32-step segments in four launches (forward states and
 * reverse segment summaries, with the forward state carried between
 * 128-step tiles by the decoupled look-back of the forward kernel; reverse
 * carries; gradients; the gw/gu reduction), k, v, gy read twice.  Otherwise
 * 16-step segments in six launches (forward segment summaries, forward
 * carries, reverse segment summaries, reverse carries, gradients, the
 * reduction), k, v read three times.  gw and gu are reduced over rows and
 * segments in a fixed order.  Results are bitwise reproducible on the
 * six-launch path and, on the four-launch path, up to two 128-step tiles;
 * beyond that reproducible to rounding (the look-back may fold the forward
 * carry from different predecessors from run to run).  Scratch (40 bytes per row, segment and channel, plus 64 bytes
 * per channel and a counter per 32 channels) is library-owned per-stream
 * memory, allocated on first use like the look-back workspace (make one call
 * of each size before stream capture).
 * No output may overlap an input or another output.  Pointers 4-byte
 * aligned.  B or T = 0 with C > 0 sets gw, gu to 0. */
WKV_API wkv_status wkv_backward(int64_t B, int64_t T, int64_t C, const float *w, const float *u,
                                const float *k, const float *v, const float *gy, float *gk,
                                float *gv, float *gw, float *gu, cudaStream_t stream);

/* The LRU's complex diagonal recurrence (review of "Resurrecting Recurrent
 * Neural Networks for Long Sequences", linear-RNN section), per complex
 * channel d:
 *
 *     x[b,t,d] = lambda_d x[b,t-1,d] + gamma_d u[b,t,d],
 *     lambda_d = e^{-nu_d + i theta_d},  nu_d = e^{nu_log[d]},  theta_d = e^{theta_log[d]}
 *
 * (the page's parameterisation: |lambda| = e^{-nu} <= 1 for any nu_log), with
 * x[b,-1,d] = x0[b,d] or 0.  u, x: [B, T, D] complex64, i.e. interleaved
 * (re, im) float pairs, [B, T, D, 2] floats; x0: [B, D] complex64 or NULL;
 * nu_log, theta_log, gamma: [D] float, gamma NULL = 1 (the page initialises
 * it to sqrt(1 - |lambda|^2)).  Pointers to complex data must be 8-byte
 * aligned (TMA path: 16-byte and D even).  lambda^n across chunk boundaries
 * is evaluated in double precision, so phases n theta of any size stay
 * exact; inside a chunk the state steps with single-precision lambda.  x must
 * not overlap an input.  Errors, streams and scratch as diag_scan. */
WKV_API wkv_status lru_scan(int64_t B, int64_t T, int64_t D, const float *nu_log,
                            const float *theta_log, const float *gamma, const float *u,
                            const float *x0, float *x, cudaStream_t stream);

/* Diagonal linear scan with bfloat16 a, b, h (fp32 h0 [B, D] or NULL; the
 * state is carried in fp32 and each h is rounded to nearest even).  Pointers
 * must be 2-byte aligned (TMA path: 16-byte and D % 8 == 0). */
WKV_API wkv_status diag_scan_bf16(int64_t B, int64_t T, int64_t D,
                                  const wkv_bf16_t *a, const wkv_bf16_t *b, const float *h0,
                                  wkv_bf16_t *h, cudaStream_t stream);

/* The gated delta rule: a linear recurrence whose state is a matrix per head
 * (the pages' recurrences keep one number per channel; this is the form their
 * successors use).  Per batch row b and value head h, with key head
 * hk = h / (HV / HK) and a_t = e^{g[b,t,h]}:
 *
 *     S' = a_t S_{t-1}                        state [DK, DV], S_{-1} = s_in or 0
 *     r_t = v[b,t,h] - S'^T k[b,t,hk]
 *     S_t = S' + beta[b,t,h] k[b,t,hk] r_t^T
 *     o[b,t,h] = scale S_t^T q[b,t,hk]
 *
 * Layout: q, k [B, T, HK, DK]; v, o [B, T, HV, DV]; g, beta [B, T, HV] float;
 * s_in, s_out [B, HV, DK, DV] float, all dense.  HK divides HV (value heads
 * share key heads in order); DK, DV are at most 128.  Where HV, DK or DV is 0
 * the call writes zeros, the sums over nothing, to every output that is not
 * NULL and not empty (o when DK is 0; of the gradients also those of the key
 * heads when HV or DV is 0).
 * g is the logarithm of the decay: g <= 0, -infinity (forget everything)
 * included.  The recurrence is a contraction for keys of length at most 1 and
 * beta in [0, 1]; other values are computed as they are.  beta = 0 and g = 0
 * leave the state as it is: how a padded batch marks its padding (with finite
 * q, k, v).  A NaN or infinity stays within its row and head, where it may
 * reach every step from the start of its 64-step chunk on.
 * s_in NULL = zeros; s_out NULL: no state out; s_out may be s_in (update in
 * place), any other overlap of an output is WKV_ERR_INVALID_ARG.  T = 0 only
 * copies the state (or zeros) to s_out.  T = 1 is one decoding step.
 * The state and every sum are fp32, whatever the I/O type.  bf16 calls that
 * take 64 steps at a time keep the operands of their products that are not
 * inputs (the state, residuals, products of keys and queries) as sums of bf16
 * parts: of all 24 bits in what reaches s_out, of 16 bits in what reaches only
 * o -- all of it when s_out is NULL, so that o may differ in the last bit of a
 * few elements from the same call with s_out.  Either way o is the rounding of a
 * value that is off by some 2^-16 of its terms' size.
 * `scratch`: caller's device memory, 16-byte aligned, at least
 * gated_delta_scratch() bytes, free to use again once the call's work on the
 * stream is done; its contents do not matter.  That is, for bf16 calls that
 * take 64 steps at a time (from 33 steps on, or 57 with more heads than SMs of
 * at most 64 columns; DK and DV multiples of 8), 33792 bytes per value head and
 * started chunk of 64 steps, 41984 with s_out; 0 (it may be NULL) for others.  Calls that may run at the same time, replays of captured graphs
 * among them, need a scratch each.  elem_bytes: 2 for the bf16 call, 4 for
 * fp32; with_state: whether s_out is given.
 * A device-side wait that gives up (of these calls and their gradients) leaves
 * NaN in every output that depends on it; wkv_device_status does not report
 * it, since they use no workspace of the library. */
WKV_API int64_t gated_delta_scratch(int64_t B, int64_t T, int64_t HV, int64_t DK, int64_t DV,
                                    int elem_bytes, int with_state);
WKV_API wkv_status gated_delta(int64_t B, int64_t T, int64_t HK, int64_t HV, int64_t DK,
                               int64_t DV, const float *q, const float *k, const float *v,
                               const float *g, const float *beta, float scale, float *o,
                               const float *s_in, float *s_out, void *scratch,
                               int64_t scratch_bytes, cudaStream_t stream);

/* gated_delta with bfloat16 q, k, v, o (fp32 g, beta and state; each o is
 * rounded once, to nearest even). */
WKV_API wkv_status gated_delta_bf16(int64_t B, int64_t T, int64_t HK, int64_t HV, int64_t DK,
                                    int64_t DV, const wkv_bf16_t *q, const wkv_bf16_t *k,
                                    const wkv_bf16_t *v, const float *g, const float *beta,
                                    float scale, wkv_bf16_t *o, const float *s_in, float *s_out,
                                    void *scratch, int64_t scratch_bytes, cudaStream_t stream);

/* Gradients of gated_delta for go = dL/do and, if not NULL, gs_out = dL/ds_out
 * [B, HV, DK, DV]: gq, gk (summed over the value heads of a key head), gv, gg,
 * gbeta and, if not NULL, gs_in = dL/ds_in.  With D_t the gradient of S_t
 * (o_t's part included), du_t = D_t^T k_t and w_t = beta_t du_t:
 *
 *     gq_t = scale S_t go_t,  gv_t = w_t,  gbeta_t = du_t . r_t,
 *     gk_t = beta_t D_t r_t - S'_t w_t,  gg_t = <D_t - k_t w_t^T, S'_t>.
 *
 * Recomputes the states from the inputs.  `scratch`: caller's device memory,
 * 16-byte aligned, at least gated_delta_backward_scratch() bytes, under the
 * same rules as gated_delta's.  That is, with T and DV rounded up to multiples
 * of 64 and 16, per value head and chunk of 64 steps 8 DV (DK + 64) bytes and,
 * for bf16 with DK and DV multiples of 8, another 100352 (DK up to 64) or
 * 124928, for others 8 DK a step (of T as it is); and up to 1 KB for alignment.
 * No output may overlap an input or another output.  T = 0: gs_in = gs_out (or
 * zeros).  Deterministic: repeated calls give the same
 * bits. */
WKV_API int64_t gated_delta_backward_scratch(int64_t B, int64_t T, int64_t HV, int64_t DK,
                                             int64_t DV, int elem_bytes);
WKV_API wkv_status gated_delta_backward(int64_t B, int64_t T, int64_t HK, int64_t HV, int64_t DK,
                                        int64_t DV, const float *q, const float *k,
                                        const float *v, const float *g, const float *beta,
                                        float scale, const float *s_in, const float *go,
                                        const float *gs_out, float *gq, float *gk, float *gv,
                                        float *gg, float *gbeta, float *gs_in, void *scratch,
                                        int64_t scratch_bytes, cudaStream_t stream);
WKV_API wkv_status gated_delta_backward_bf16(int64_t B, int64_t T, int64_t HK, int64_t HV,
                                             int64_t DK, int64_t DV, const wkv_bf16_t *q,
                                             const wkv_bf16_t *k, const wkv_bf16_t *v,
                                             const float *g, const float *beta, float scale,
                                             const float *s_in, const wkv_bf16_t *go,
                                             const float *gs_out, wkv_bf16_t *gq, wkv_bf16_t *gk,
                                             wkv_bf16_t *gv, float *gg, float *gbeta,
                                             float *gs_in, void *scratch, int64_t scratch_bytes,
                                             cudaStream_t stream);

/* Test hook for the bounded waits of the gated delta rule's bf16 kernels over
 * chunks of 64 steps, process-wide, for later launches.  kernel 1 (preparation
 * of the chunks), 2 (the chain of the states) or 3 (gradients within a chunk)
 * does not make chunk `chunk`'s copies (2: nor any after it in its direction),
 * so the waits for them run out, after 2 seconds.  The outcome is NaN in the
 * outputs that depend on the chunk; the context stays usable.  (0, 0) turns it
 * off.  WKV_ERR_INVALID_ARG for values out of range. */
WKV_API wkv_status gated_delta_set_fault_injection(int kernel, int chunk);

/* Group norm with an activation, channels last: the normalisation and gate
 * between a recurrence over heads and the output projection.  Each of N tokens
 * (rows of C channels) is normalised on its own, in `groups` groups of
 * D = C / groups consecutive channels (statistics never cross tokens):
 *
 *     n = (x - mean) / sqrt(var + eps),  h = n weight + bias,
 *     y = h act(gate),  or act(h) when gate is NULL,
 *
 * var the biased variance; act(z) = z, z / (1 + e^{-z}) or 1 / (1 + e^{-z}).
 * x, gate, y: [N, C]; weight, bias: [C] float or NULL (1 and 0).  groups
 * divides C, D <= 4096, eps >= 0.  y must not overlap an input. */
typedef enum { WKV_ACT_NONE = 0, WKV_ACT_SILU = 1, WKV_ACT_SIGMOID = 2 } wkv_activation;
WKV_API wkv_status group_norm(int64_t N, int64_t C, int64_t groups, const float *x,
                              const float *weight, const float *bias, const float *gate, int act,
                              float eps, float *y, cudaStream_t stream);

/* group_norm with bfloat16 x, gate, y (fp32 weight, bias; computed in fp32 and
 * rounded once, to nearest even). */
WKV_API wkv_status group_norm_bf16(int64_t N, int64_t C, int64_t groups, const wkv_bf16_t *x,
                                   const float *weight, const float *bias, const wkv_bf16_t *gate,
                                   int act, float eps, wkv_bf16_t *y, cudaStream_t stream);

/* Gradients of group_norm for gy = dL/dy: gx, ggate (given exactly when gate
 * is) and, if not NULL, gweight and gbias [C], summed over the tokens in a
 * fixed order.  With gh = gy act(gate) (or gy act'(h)) and gn = gh weight:
 *
 *     gx = (gn - mean(gn) - n mean(gn n)) / sqrt(var + eps),
 *     ggate = gy h act'(gate),  gweight = sum gh n,  gbias = sum gh.
 *
 * `scratch`: caller's device memory, 16-byte aligned, at least
 * group_norm_backward_scratch() bytes, under the same rules as
 * gated_delta_backward's.  N = 0 sets gweight and gbias to 0. */
WKV_API int64_t group_norm_backward_scratch(int64_t N, int64_t C);
WKV_API wkv_status group_norm_backward(int64_t N, int64_t C, int64_t groups, const float *x,
                                       const float *weight, const float *bias, const float *gate,
                                       int act, float eps, const float *gy, float *gx,
                                       float *gweight, float *gbias, float *ggate, void *scratch,
                                       int64_t scratch_bytes, cudaStream_t stream);
WKV_API wkv_status group_norm_backward_bf16(int64_t N, int64_t C, int64_t groups,
                                            const wkv_bf16_t *x, const float *weight,
                                            const float *bias, const wkv_bf16_t *gate, int act,
                                            float eps, const wkv_bf16_t *gy, wkv_bf16_t *gx,
                                            float *gweight, float *gbias, wkv_bf16_t *ggate,
                                            void *scratch, int64_t scratch_bytes,
                                            cudaStream_t stream);

/* WKV forward, fp32, without allocating any device memory.  The pages this
 * library follows have no counterpart of this entry point: it exists for
 * callers that cannot call cudaMalloc -- code running inside an engine that
 * has already reserved the GPU's memory for its own pool, plugin interfaces
 * that hand an operator nothing but its input and output buffers, and
 * latency-critical paths that must not pay for an allocation or for the
 * device-wide synchronisation cudaMalloc / cudaFree can cause.
 *
 * Same operation, arguments, layout and host-side checks as wkv_forward.
 * Instead of a workspace, the state passed between thread blocks lives in one
 * fixed 16 MiB device array; every GPU that uses this entry point holds it
 * from its first call until the process exits.  A problem whose scratch would
 * not fit -- more than 32,767 tiles, i.e. B * ceil(C/32) * ceil(T/128) >
 * 32,767 (sequences of at most 128 steps need no scratch) -- is rejected with
 * WKV_ERR_INVALID_ARG before anything runs; use wkv_forward for it.
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current) and sets kernel
 * attributes; make that first call before any stream capture.
 * Every call on a device shares the one array and first clears (cudaMemsetAsync
 * on `stream`) the counters and records that must start at zero, so calls whose
 * work overlaps on the GPU -- on different streams, or from several host
 * threads -- race and give wrong results: serialise them.  A device-side wait
 * that gives up leaves NaN in the affected outputs; wkv_device_status does not
 * report it for this entry point. */
WKV_API wkv_status wkv_forward_noalloc(int64_t B, int64_t T, int64_t C,
                                       const float *w, const float *u,
                                       const float *k, const float *v, float *y,
                                       cudaStream_t stream);

/* The same three operations on HOST buffers (every pointer, w/u/h0 included,
 * is host memory; NULL h0 = zeros).  The call copies the inputs to the
 * device, runs the kernel and copies the outputs back, and returns when they
 * are in the output buffer (synchronous; no stream argument).  The work is cut
 * into up to 8 independent chunks of at least 16 MB of input -- batch rows, or
 * 64-channel-aligned channel slices when B is 1 -- pipelined over three
 * internal streams so the uploads of one chunk overlap the compute and
 * download of another.  Page-locked host
 * memory (cudaHostAlloc / cudaHostRegister) gives full overlap; pageable memory
 * works but its copies are staged by the driver.  The library allocates device
 * staging (three chunks of inputs, outputs and parameters) on first use and
 * grows it on demand.  Calls are serialised across host threads.  Returns
 * WKV_ERR_TIMEOUT if a device-side wait gave up during the call. */
WKV_API wkv_status wkv_forward_host(int64_t B, int64_t T, int64_t C,
                                    const float *w, const float *u,
                                    const float *k, const float *v, float *y);
WKV_API wkv_status wkv_forward_bf16_host(int64_t B, int64_t T, int64_t C,
                                         const float *w, const float *u,
                                         const wkv_bf16_t *k, const wkv_bf16_t *v,
                                         wkv_bf16_t *y);
WKV_API wkv_status diag_scan_host(int64_t B, int64_t T, int64_t D,
                                  const float *a, const float *b, const float *h0, float *h);

/* Synchronise `stream`, then return and clear the device status word of that
 * stream's workspace: WKV_OK, or WKV_ERR_TIMEOUT if a device-side wait gave up
 * since the last query.  WKV_ERR_CUDA if the synchronisation itself failed. */
WKV_API wkv_status wkv_device_status(cudaStream_t stream);

/* Message for the last non-OK return on the calling thread ("" if none). */
WKV_API const char *wkv_last_error(void);

/* Free every workspace the library holds on the current device (synchronises
 * the device first).  Later calls allocate again on demand. */
WKV_API wkv_status wkv_release_workspaces(void);

/* Tuning knob, process-wide: the number of steps one thread block stages per
 * tile (8, 32, 64, 128 or 256), or 0 (the default) to let each call choose:
 * 128, or 256 for sequences longer than 4096 steps whose rows and channels
 * make fewer than 64 tiles per tile-length of time.  Results do not depend on
 * it beyond rounding: it only moves the boundaries where chunk summaries are
 * combined.  WKV_ERR_INVALID_ARG for any other value. */
WKV_API wkv_status wkv_set_tile_steps(int steps);
WKV_API int wkv_get_tile_steps(void);
/* The tile length a WKV or scan call of this shape uses now (elem_bytes: 4
 * for fp32 I/O, 2 for bf16); 0 for an invalid shape. */
WKV_API int wkv_tile_steps_for(int64_t B, int64_t T, int64_t C, int elem_bytes);

/* Test hook for failure detection, process-wide, for later launches of the
 * allocating entry points.  skip_tile >= 0: that tile (in the launch's
 * ticket numbering) never publishes its state, so the bounded look-back waits
 * of the tiles after it in time run out; spin_limit > 0 replaces the number
 * of polls a wait makes before giving up (0 restores the default, about a
 * second).  The outcome is WKV_ERR_TIMEOUT from wkv_device_status and NaN in
 * the affected outputs; the context stays usable.  (-1, 0) turns it off.
 * WKV_ERR_INVALID_ARG for skip_tile < -1 or spin_limit < 0. */
WKV_API wkv_status wkv_set_fault_injection(int skip_tile, long long spin_limit);

#ifdef __cplusplus
}
#endif

#endif /* WKV_B200_H */
