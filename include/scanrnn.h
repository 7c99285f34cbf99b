/*
 * scanrnn.h -- C ABI of the MI355X (gfx950) minGRU / MinMax scan library.
 *
 * What the calls compute
 * ----------------------
 * minGRU layer (the log-space minGRU layer profiled on openvist.com as
 * "Mingru Pytorch"; intro and "Requirements & limits": a log-space numerically
 * stable layer with a parallel mode and a token-by-token mode that carries the
 * hidden state):
 *
 *     [k_t | p_t] = x_t W_in                 (k: first D_h columns, p: next D_h)
 *     z_t = sigma(k_t),   htilde_t = g(p_t),  g(v) = v + 1/2 (v >= 0), sigma(v) (v < 0)
 *     h_t = (1 - z_t) h_{t-1} + z_t htilde_t       t = 1..T, h_0 carried (absent = 0)
 *     y_t = h_t W_out                        (absent W_out: y_t = h_t)
 *
 * evaluated as an associative scan over t of the affine maps
 * h -> a_t h + b_t.  The log-space coefficients log a_t = log(1 - z_t) =
 * -softplus(k_t) and log b_t = log z_t + log g(p_t) are exponentiated in
 * closed form (a_t = sigma(-k_t), b_t = sigma(k_t) g(p_t), no cancelling
 * 1 - x), and composed maps carry their coefficient A together with its
 * complement 1 - A, so that a long memory (A near 1) keeps 1 - A to a few
 * ulps -- what the log-space form's -softplus(k) keeps -- while the state
 * itself stays linear (a signed h_0 needs no logarithm).  The single-token
 * step evaluates h_{t-1} + z_t (g(p_t) - h_{t-1}).
 *
 * Range.  For |k| above about 87.3 the smaller of sigma(k) and sigma(-k) is
 * below the smallest normal fp32 number and flushes to zero, and the term it
 * multiplies (the candidate's share for very negative k, the carried state
 * for very positive k) is dropped; every other term keeps full accuracy.
 * The scans report such gate logits through scanrnn_workspace_status
 * (SR_ERR_GATE_RANGE); the results are still written.
 *
 * MinMax neuron (minmaxrnc PyPI page, "The model" item 3):
 *
 *     x_{t+1} = max(min(r_t, x_t), s_t)   element-wise, by a prefix scan.
 *
 * Conventions shared by every call
 * --------------------------------
 * - All tensor pointers are DEVICE pointers; the caller owns every buffer,
 *   including the workspace.  The library keeps no pointer after a call
 *   returns and holds no global mutable state except a thread-local error
 *   string, the look-back poll bound (scanrnn_set_lookback_spin_limit) and
 *   the device array of mingru_scan_noalloc (with the caller-owned-buffer
 *   rule its one exception).
 * - Tensors are row-major, innermost (feature) dimension fastest; a [B,T,D]
 *   tensor is B*T rows of D elements.  Pointers must be aligned to their
 *   element size; wider alignment (8 or 16 bytes) lets the library use
 *   vector loads.
 * - Sizes are int64.  B*T*D may exceed 2^31; offsets are computed in 64 bits.
 * - Calls are asynchronous on `stream` (a hipStream_t; NULL = the default
 *   stream).  Buffers must stay alive until the enqueued work completes.
 * - Arguments are validated before anything is enqueued: on any non-OK status
 *   nothing was launched and no output was written.  A failed HIP launch
 *   returns SR_ERR_HIP.  scanrnn_last_error() gives the text of the last
 *   non-OK status on the calling thread.  No C++ exception crosses the ABI.
 * - Calls are reentrant; concurrent calls must use distinct workspaces.
 * - Workspace: at least *_workspace_size(...) bytes, 256-byte aligned,
 *   contents need not be initialised (the call resets what it uses, on the
 *   stream, before the scan).
 * - Determinism: minmax_scan is bit-exact (min and max only select).  The
 *   minGRU calls agree with the sequential definition within rounding; the
 *   order in which partial results are combined does not depend on timing,
 *   so repeated calls give identical bits.
 */
#ifndef SCANRNN_H
#define SCANRNN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SR_OK = 0,
  SR_ERR_INVALID_ARGUMENT = 1,   /* null pointer, negative size, bad stride     */
  SR_ERR_UNSUPPORTED = 2,        /* valid request the library does not handle   */
  SR_ERR_WORKSPACE_TOO_SMALL = 3,
  SR_ERR_HIP = 4,                /* a HIP runtime call failed                   */
  SR_ERR_LOOKBACK_TIMEOUT = 5,   /* reported by scanrnn_workspace_status only   */
  SR_ERR_GATE_RANGE = 6          /* reported by scanrnn_workspace_status only   */
} sr_status;

/* Element type of k and p: one of these values, passed as a 32-bit integer
 * so that whatever a caller sends is a valid value of the type; any other
 * value is rejected with SR_ERR_INVALID_ARGUMENT. */
enum { SR_F32 = 0, SR_BF16 = 1 };
typedef int32_t sr_dtype;

/* Bytes of workspace mingru_forward needs.  has_w_in / has_w_out say whether
 * the call will pass W_in / W_out.  W_out needs B*T*D_h floats to stage h.
 * With W_in, large problems (at least 512 tiles of 256 steps x 64 channels)
 * compute the projection inside the scan and need no more; smaller ones
 * stage [k|p] (B*T*2*D_h floats) and split-K partial sums. */
size_t mingru_forward_workspace_size(int64_t B, int64_t T, int64_t D_in, int64_t D_h,
                                     int64_t D_out, int has_w_in, int has_w_out);

/*
 * Parallel mode: the whole sequence at once (minGRU profile, guide "Install
 * and apply the minGRU layer": the output has the input's shape).
 *
 *   x      [B,T,D_in] fp32; read only when W_in != NULL.
 *   W_in   [D_in, 2*D_h] fp32, or NULL: then k and p are given directly
 *          (scan-only use) and x must be NULL.
 *   k, p   rows of the pre-projected gate logits / candidate pre-activations,
 *          element (b,t,d) at k[(b*T + t)*ld_kp + d]; dtype kp_dtype
 *          (SR_F32 or SR_BF16).  ld_kp >= D_h, so k and p may be the two
 *          halves of one [B,T,2*D_h] buffer.  Used only when W_in == NULL.
 *   h0     [B,D_h] fp32 carried state, or NULL (zero state).
 *   W_out  [D_h, D_out] fp32, or NULL (then D_out must equal D_h, y = h).
 *   y      [B,T,D_out] fp32 output.
 *   h_last [B,D_h] fp32, or NULL: receives h_T (h0, or zeros, when T == 0).
 */
sr_status mingru_forward(int64_t B, int64_t T, int64_t D_in, int64_t D_h, int64_t D_out,
                         const float* x, const float* W_in,
                         const void* k, const void* p, int64_t ld_kp, sr_dtype kp_dtype,
                         const float* h0, const float* W_out,
                         float* y, float* h_last,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace mingru_step needs: none up to 512 streams, nor up to
 * 4096 streams while D_in and D_h are at most 1024 (the K range is then
 * split inside each workgroup); otherwise split-K partial sums. */
size_t mingru_step_workspace_size(int64_t B, int64_t D_in, int64_t D_h, int64_t D_out);

/*
 * Sequential mode, one token (minGRU profile, guide "Process a sequence
 * sequentially with carried hidden state"; the minGRU tutorial's Step 3: the
 * base step returns the new hidden state, which is also its output).
 *
 *   x_t    [B,D_in] fp32;  W_in [D_in,2*D_h] fp32 (required).
 *   W_out  [D_h,D_out] fp32 or NULL (then D_out must equal D_h).
 *   h_prev [B,D_h] fp32 or NULL (zero state).
 *   h_next [B,D_h] fp32; may be the same buffer as h_prev.
 *   y_t    [B,D_out] fp32, or NULL when W_out is NULL (the output is h_next;
 *          a non-NULL y_t then receives a copy).
 */
sr_status mingru_step(int64_t B, int64_t D_in, int64_t D_h, int64_t D_out,
                      const float* x_t, const float* W_in, const float* W_out,
                      const float* h_prev, float* h_next, float* y_t,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * Time decay of the carried state (the decay contract of the minGRU tutorial
 * "Your first delta model", Step 5 "Adding time decay": each event comes with
 * the gap delta_t preceding it; the carried state is scaled by gamma once per
 * token, at the token boundary, before that token's own write; a zero gap is
 * gamma = exp(0) = 1; a rate * gap above about 1e4 saturates float32 and
 * wipes the memory, through a clamp, and is reported; log1p_delta compresses
 * the gaps).  On the minGRU's vector state:
 *
 *     gap_t  = log1p(delta_t) if log1p_delta else delta_t
 *     gamma  = exp(-min(decay_rate_d * gap_t, 1e4))
 *     h_t    = (1 - z_t) (gamma_t h_{t-1}) + z_t g(p_t)
 *
 *   decay_rate  [D_h] fp32 per-channel rate, >= 0 and finite.
 *   delta_t     [B,T] fp32 (sequence call) or [B] (step), contiguous, >= 0
 *               and finite.  Other values are outside the contract.
 *   log1p_delta 0 or 1.
 *   saturated   device uint32 or NULL: set to 1 (atomic OR, never cleared by
 *               the library) when some decay_rate_d * gap_t, rounded to fp32,
 *               exceeds 1e4.  exp(-1e4) is 0 in fp32, so the clamp changes no
 *               value; the flag says large gaps were not distinguished.
 *
 * Everything else is as in mingru_forward / mingru_step, with the same
 * workspace sizes (mingru_forward_workspace_size, mingru_step_workspace_size).
 */
sr_status mingru_forward_decayed(int64_t B, int64_t T, int64_t D_in, int64_t D_h, int64_t D_out,
                                 const float* x, const float* W_in,
                                 const void* k, const void* p, int64_t ld_kp, sr_dtype kp_dtype,
                                 const float* decay_rate, const float* delta_t, int log1p_delta,
                                 uint32_t* saturated,
                                 const float* h0, const float* W_out,
                                 float* y, float* h_last,
                                 void* workspace, size_t workspace_bytes, void* stream);

sr_status mingru_step_decayed(int64_t B, int64_t D_in, int64_t D_h, int64_t D_out,
                              const float* x_t, const float* W_in, const float* W_out,
                              const float* decay_rate, const float* delta_t, int log1p_delta,
                              uint32_t* saturated,
                              const float* h_prev, float* h_next, float* y_t,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace minmax_scan needs. */
size_t minmax_scan_workspace_size(int64_t B, int64_t T, int64_t D);

/*
 * MinMax neuron over a sequence (minmaxrnc PyPI page, "The model" item 3;
 * "Quick start" carries the state across calls).
 *
 *   r, s   [B,T,D] fp32 inputs of steps t = 0..T-1.
 *   x0     [B,D] fp32 initial state (required).
 *   x_out  [B,T,D] fp32: x_out[:,t,:] = x_{t+1}.
 *   x_last [B,D] fp32 or NULL: receives x_T (x0 when T == 0).
 * Results are bit-exact; NaN inputs are outside the contract.
 */
sr_status minmax_scan(int64_t B, int64_t T, int64_t D,
                      const float* r, const float* s, const float* x0,
                      float* x_out, float* x_last,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * One MinMax step for a single token, O(1) work and O(D) memory per token
 * (minmaxrnc page, "Key properties": efficient inference as a true RNN;
 * "Quick start": generation steps one token at a time carrying the state):
 *     x_next = max(min(r_t, x_prev), s_t)   element-wise over [B, D].
 * x_next may be the same buffer as x_prev.  No workspace.  Bit-exact.
 */
sr_status minmax_step(int64_t B, int64_t D, const float* r_t, const float* s_t,
                      const float* x_prev, float* x_next, void* stream);

/* Bytes of workspace the backward calls need. */
size_t mingru_scan_backward_workspace_size(int64_t B, int64_t T, int64_t D);
size_t minmax_scan_backward_workspace_size(int64_t B, int64_t T, int64_t D);

/*
 * Backward pass of the minGRU scan (the layers are trained: minGRU profile,
 * "Requirements & limits", training entry point).  For L with dL/dh_t = dh
 * on every output h_t (the scan-only mingru_forward's y) and dL/dh_T =
 * dh_last, returns
 *     dk_t = G_t z_t (1 - z_t) (g(p_t) - h_{t-1}),  dp_t = G_t z_t g'(p_t),
 *     dh0  = (1 - z_1) G_1,   with  G_t = dh_t + (1 - z_{t+1}) G_{t+1}.
 *
 *   k, p     the forward inputs (rows of ld_kp elements, kp_dtype).
 *   h0       [B,D] forward initial state or NULL (zero).
 *   h        [B,T,D] fp32 forward outputs h_1..h_T.
 *   dh       [B,T,D] fp32 upstream gradient;  dh_last [B,D] or NULL.
 *   dk, dp   [B,T,D] fp32 outputs (contiguous).  dh0 [B,D] or NULL.
 */
sr_status mingru_scan_backward(int64_t B, int64_t T, int64_t D,
                               const void* k, const void* p, int64_t ld_kp, sr_dtype kp_dtype,
                               const float* h0, const float* h, const float* dh,
                               const float* dh_last, float* dk, float* dp, float* dh0,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward pass of the time-decayed minGRU scan (mingru_forward_decayed
 * without projections; decay contract of the delta tutorial, Step 5
 * "Adding time decay").  With gamma_t = exp(-min(decay_rate_d * gap_t, 1e4))
 * and c_t = (1 - z_t) gamma_t:
 *     dk_t = G_t z_t (1 - z_t) (g(p_t) - gamma_t h_{t-1}),  dp_t = G_t z_t g'(p_t),
 *     dh0  = c_1 G_1,   with  G_t = dh_t + c_{t+1} G_{t+1}.
 * decay_rate [D], delta_t [B,T] and log1p_delta as in mingru_forward_decayed
 * (the rates and gaps get no gradient); everything else and the workspace
 * size (mingru_scan_backward_workspace_size) as in mingru_scan_backward.
 */
sr_status mingru_scan_backward_decayed(int64_t B, int64_t T, int64_t D,
                                       const void* k, const void* p, int64_t ld_kp,
                                       sr_dtype kp_dtype,
                                       const float* decay_rate, const float* delta_t,
                                       int log1p_delta,
                                       const float* h0, const float* h, const float* dh,
                                       const float* dh_last, float* dk, float* dp, float* dh0,
                                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward pass of the MinMax scan (minmaxrnc page, "Key properties": the
 * gradient through the state path neither vanishes nor explodes -- it is
 * routed, unchanged, to the operand each step selects).  Gradients dx on
 * x_out and dx_last on x_T; r, s, x0 and x_out are the forward's.  Ties
 * (measure zero) route to the state: s only if strictly above min(r, x),
 * r only if strictly below x.  dr, ds [B,T,D], dx0 [B,D] or NULL.
 */
sr_status minmax_scan_backward(int64_t B, int64_t T, int64_t D,
                               const float* r, const float* s, const float* x0,
                               const float* x_out, const float* dx, const float* dx_last,
                               float* dr, float* ds, float* dx0,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * The scan-only mingru_forward (W_in and W_out NULL, y = h) for callers that
 * cannot allocate -- code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc: no workspace argument and no allocation
 * of any kind.  Its look-back words live in a fixed device array of
 * mingru_scan_noalloc_max_workspace() bytes (32 MiB), one per GPU, held
 * until the process ends; requests needing more (scan workspace above that:
 * B * ceil(T/144) * D * 8 + 256 bytes) return SR_ERR_UNSUPPORTED before any
 * HIP call.  Every call on a GPU shares that GPU's array and resets it
 * first, on `stream`: calls in one stream are ordered and safe, calls that
 * overlap on one GPU (several streams, several host threads) race.  Results
 * are those of mingru_forward on the same inputs, bit for bit.  The first
 * call on a device looks up that device's copy of the array.
 *
 *   k, p, ld_kp, kp_dtype, h0   as in mingru_forward (scan-only use).
 *   h       [B,T,D] fp32 output;  h_last [B,D] fp32 or NULL.
 */
size_t mingru_scan_noalloc_max_workspace(void);
sr_status mingru_scan_noalloc(int64_t B, int64_t T, int64_t D,
                              const void* k, const void* p, int64_t ld_kp, sr_dtype kp_dtype,
                              const float* h0, float* h, float* h_last, void* stream);

/*
 * 8-bit codes: symmetric, one fp32 scale per row.
 *
 *     scale = max |x| / 127,   q = rint(x / scale) in [-127, 127]
 *
 * (two IEEE fp32 divisions, ties to even).  A row of zeros has scale 0 and
 * codes 0; a row holding a NaN or an infinity has scale NaN and codes 0, so
 * that every product with it is NaN.  Codes are stored as contiguous rows of
 * quantized_row_bytes(K) = K rounded up to 128 bytes, zeros behind the K
 * codes (the products read whole 128-byte lines; zeros add nothing).
 *
 * quantize_rows: the rows of x [M,K] (a token's activations each), rows of
 *   ldx >= K elements, x_dtype SR_F32 or SR_BF16 -> q [M, quantized_row_bytes(K)],
 *   scale [M].
 * quantize_columns: the columns of W [K,N] (rows of ldw >= N elements; an
 *   output channel each) -> q [N, quantized_row_bytes(K)], transposed, scale [N].
 * q must be 16-byte aligned.  K = 0 gives scales 0 and no codes.  More than
 * 16777215 rows (quantize_columns: columns) are SR_ERR_UNSUPPORTED.
 */
int64_t quantized_row_bytes(int64_t K);
sr_status quantize_rows(int64_t M, int64_t K, const void* x, int64_t ldx, sr_dtype x_dtype,
                        int8_t* q, float* scale, void* stream);
sr_status quantize_columns(int64_t K, int64_t N, const void* W, int64_t ldw, sr_dtype w_dtype,
                           int8_t* q, float* scale, void* stream);

/*
 * Product of codes with a scale per token and per output channel:
 *
 *     y[m, n] = (sum_k a[m, k] b[n, k]) (a_scale[m] b_scale[n])
 *
 * The sum is exact (32-bit integers); it is rounded once to fp32, scaled, and
 * rounded once more when y is bf16.  Results do not depend on the order of
 * anything, so repeated calls give identical bits.
 *
 *   K       stored width of both operands: a multiple of 128, at most 131072
 *           (larger: SR_ERR_UNSUPPORTED; 127^2 K must stay below 2^31).
 *   a, b    [M,K] and [N,K] codes in [-127, 127], rows of lda / ldb >= K
 *           bytes; a, b, lda and ldb multiples of 16.
 *   y       [M,N] in y_dtype, rows of ldy >= N elements.
 * SR_ERR_UNSUPPORTED: M or N above 16777215, M N above about 2^38, rows of
 * codes more than 8 MiB apart.
 */
sr_status matmul_i8(int64_t M, int64_t N, int64_t K, const int8_t* a, int64_t lda,
                    const float* a_scale, const int8_t* b, int64_t ldb, const float* b_scale,
                    void* y, int64_t ldy, sr_dtype y_dtype, void* stream);

/*
 * mingru_step and mingru_forward on 8-bit weights: the activations are
 * quantised row by row (x before W_in, h before W_out), the products run on
 * codes, and the recurrence stays in fp32.
 *
 *   x_t, x        as in mingru_step / mingru_forward, x_dtype SR_F32 or SR_BF16.
 *   W_in          [2*D_h, quantized_row_bytes(D_in)] codes and W_in_scale [2*D_h]
 *                 of the fp32 W_in's columns (quantize_columns).
 *   W_out         [D_out, quantized_row_bytes(D_h)] codes and W_out_scale [D_out],
 *                 or NULL (both; then D_out must equal D_h).
 *   decay_rate    NULL (no time decay; delta_t and saturated must then be NULL),
 *                 or as in mingru_step_decayed / mingru_forward_decayed with delta_t,
 *                 log1p_delta and saturated.
 *   y_t           [B,D_out] in x_dtype.  Without W_out the output is h_next and
 *                 y_t must be NULL.
 *   y             [B,T,D_out] in x_dtype; without W_out the states h, in fp32.
 * mingru_forward_i8 hands [k|p] to the scan in x_dtype: with bf16 activations
 * the gates are rounded to bf16, which halves the staged bytes and is below
 * the rounding of the 8-bit codes.  Everything else as in mingru_step / mingru_forward;
 * codes 16-byte aligned; D_in and D_h at most 131072, W_in below 4 GiB, B (times T)
 * at most 16777215 (else SR_ERR_UNSUPPORTED).
 * mingru_step_i8: h_next may be the same buffer as h_prev; otherwise it must not
 * overlap h_prev, and it must never overlap x_t or y_t (each is refused with
 * SR_ERR_INVALID_ARGUMENT).  A row's results do not depend on the rows beside it.
 */
size_t mingru_step_i8_workspace_size(int64_t B, int64_t D_in, int64_t D_h, int64_t D_out);
sr_status mingru_step_i8(int64_t B, int64_t D_in, int64_t D_h, int64_t D_out,
                         const void* x_t, sr_dtype x_dtype,
                         const int8_t* W_in, const float* W_in_scale,
                         const int8_t* W_out, const float* W_out_scale,
                         const float* decay_rate, const float* delta_t, int log1p_delta,
                         uint32_t* saturated,
                         const float* h_prev, float* h_next, void* y_t,
                         void* workspace, size_t workspace_bytes, void* stream);

size_t mingru_forward_i8_workspace_size(int64_t B, int64_t T, int64_t D_in, int64_t D_h,
                                        int64_t D_out, sr_dtype x_dtype, int has_w_out);
sr_status mingru_forward_i8(int64_t B, int64_t T, int64_t D_in, int64_t D_h, int64_t D_out,
                            const void* x, sr_dtype x_dtype,
                            const int8_t* W_in, const float* W_in_scale,
                            const int8_t* W_out, const float* W_out_scale,
                            const float* decay_rate, const float* delta_t, int log1p_delta,
                            uint32_t* saturated,
                            const float* h0, void* y, float* h_last,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * One AdamW step over many tensors, few launches whatever their number.  For
 * each element, t = step >= 1, c1 = 1 - beta1^t, c2 = 1 - beta2^t:
 *
 *     g = grad * grad_scale
 *     m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *     p = p (1 - lr weight_decay) - (lr / c1) m / (sqrt(v) / sqrt(c2) + eps)
 *
 * in fp32; a bf16 p is rounded once.  In place on params and states.
 *
 *   tensors     n_tensors descriptions in HOST memory, read before the call
 *               returns.  A tensor with grad NULL is left as it is, states
 *               included.  param and grad are contiguous and aligned to their
 *               element sizes.  No two params of a step may share memory (tied
 *               weights are one tensor: SR_ERR_INVALID_ARGUMENT).
 *   m, v        device states of all tensors one after another, each tensor's span
 *               rounded up to 256 elements (adamw_state_elements(n)); state_elements
 *               is their length, at least the sum of the spans.  16-byte aligned.
 *   state_bits  32: fp32 m and v; m_scale and v_scale must be NULL.
 *               8: m and v hold one float8 e4m3 (OCP) code per element, of m and
 *               of sqrt(v), each block of 256 elements with one fp32 scale in m_scale /
 *               v_scale [state_elements / 256]: value = code * scale, scale = the
 *               block's largest magnitude times the fp32 nearest to 1 / 448, codes to
 *               nearest; a positive sqrt(v)
 *               never gets the code 0 (it is raised to 2^-9).  A block whose state
 *               holds a NaN or an infinity gets the scale NaN.  Zeroed buffers are
 *               the states before the first step.
 *               Limit of the 8-bit v: its codes are 6 to 12 % apart, and one step
 *               moves sqrt(v) by less (by (1 - beta2) / 2 where a gradient stops), so
 *               an element follows its block's largest one, which is held exactly.
 *               While the gradients of a block keep their proportions, sqrt(v) stays
 *               within about 0.7 to 1.7 of its fp32 value.  An element whose gradients
 *               shrink against the rest of its block keeps its old sqrt(v), or rises
 *               with the block, and its steps are too small by that factor; one whose
 *               gradients grow falls behind by up to about 8 times (beta2 = 0.999;
 *               3 times with 0.99), with steps too large by that.  beta2 below about
 *               0.88 follows.  Use 32 bits where single elements change like that.
 *   grad_scale  device fp32 scalar multiplied onto every gradient (clipping, loss
 *               scaling), or NULL.
 * The step and the hyperparameters travel with the launch: a captured graph
 * replays those of its capture.
 *
 * adamw_step_each: the same with a step number of its own for each tensor,
 * steps[i] >= 1 in HOST memory (read before the call returns; not read where
 * grad is NULL).  A tensor whose first gradient comes late, or that is left out of
 * some steps, counts its own: its states start from zero then, and the
 * corrections by c1 and c2 belong to them.
 */
typedef struct {
  void* param;
  const void* grad;
  int64_t n;               /* elements */
  sr_dtype param_dtype;    /* SR_F32 or SR_BF16 */
  sr_dtype grad_dtype;
} sr_adamw_tensor;

int64_t adamw_state_elements(int64_t n);
sr_status adamw_step(int64_t n_tensors, const sr_adamw_tensor* tensors, void* m, void* v,
                     float* m_scale, float* v_scale, int state_bits, int64_t state_elements,
                     int64_t step, double lr, double beta1, double beta2, double eps,
                     double weight_decay, const float* grad_scale, void* stream);
sr_status adamw_step_each(int64_t n_tensors, const sr_adamw_tensor* tensors, void* m, void* v,
                          float* m_scale, float* v_scale, int state_bits, int64_t state_elements,
                          const int64_t* steps, double lr, double beta1, double beta2, double eps,
                          double weight_decay, const float* grad_scale, void* stream);

/*
 * Selective state space scan (input-dependent steps and a state of N numbers
 * per channel), the short causal convolution in front of it and the norm with the
 * residual's addition around them.  What the five calls of the scan and the
 * convolution share:
 *
 *   lengths     device int32 [B] or NULL: tokens of each sequence of a padded batch
 *               (values outside [0, T] count as the nearer end).  What stands behind a
 *               sequence's end is not read into any result, whatever its values;
 *               outputs and gradients there are zeros, and the last state is the
 *               one behind the sequence's last token (the first state where it
 *               has none).
 *   ld_*        distance of the rows (b, t) of a tensor in elements, row b*T + t at
 *               (b*T + t) * ld: halves of one projection's output are rows of it.
 *   outputs     contiguous.  They must not overlap inputs or each other
 *               (SR_ERR_INVALID_ARGUMENT).
 * Repeated calls of equal sizes give identical bits (a sequence alone may be cut
 * otherwise than in a batch, and differ by roundings).  No call allocates, waits for the GPU or
 * keeps anything; all can be captured into a graph.  Sizes whose launches would
 * take 2^32 work-items or more are SR_ERR_UNSUPPORTED.
 *
 * selective_scan_forward:
 *
 *     dt_t = softplus(delta_t + delta_bias)     (delta_softplus 0: delta_t + delta_bias)
 *     h_n  = exp(dt_t A_n) h_n + dt_t u_t B_tn          n = 1..N, per channel
 *     y_t  = (sum_n C_tn h_n + skip u_t) silu(z_t)
 *
 *   u, delta, z   [B,T,D] rows in x_dtype (SR_F32 or SR_BF16); z NULL: no gate.
 *   Bm, Cm        [B,T,G,N] rows in x_dtype: G groups of D/G neighbouring channels
 *                 that share them.  G divides D.
 *   A             [D,N] fp32, usually negative.
 *   skip, delta_bias  [D] fp32 or NULL (zeros).
 *   h0, h_last    [B,D,N] fp32 state in front of and behind the tokens; NULL: zeros,
 *                 and not wanted.
 *   y             [B,T,D] in x_dtype.
 * States, steps and gates are fp32; y is rounded once.  N at most 64, rows of
 * several tokens at most 2^25 elements apart (else SR_ERR_UNSUPPORTED).  Few channels
 * and long sequences are cut into chunks of tokens whose decay is the exponential of
 * their summed steps; a state that left the fp32 range stays non-finite, but may
 * become NaN where one token after the other would give an infinity.  The gradients
 * that an infinite input or state goes into may be NaN where the formula gives an infinity;
 * other channels', sequences' and groups' stay as they are.
 *
 * selective_scan_backward: for dL/dy = dy and dL/dh_last = dh_last (or NULL), the
 * gradients of u, delta, z, Bm and Cm in x_dtype (dB and dC summed over the
 * channels of a group), of A, skip, delta_bias and h0 in fp32.  dz goes with z;
 * dskip, ddelta_bias and dh0 may be NULL.  The states are computed again.
 *
 * selective_step: one token, rows [B,D] and [B,G,N]; h_next may be the same buffer
 * as h_prev (NULL: zeros), else they must not overlap.
 */
size_t selective_scan_forward_workspace_size(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G);
sr_status selective_scan_forward(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, const void* u,
                         int64_t ld_u, const void* delta, int64_t ld_delta, const void* z,
                         int64_t ld_z, const void* Bm, int64_t ld_b, const void* Cm, int64_t ld_c,
                         sr_dtype x_dtype, const float* A, const float* skip,
                         const float* delta_bias, int delta_softplus, const float* h0,
                         const int32_t* lengths, void* y, float* h_last, void* workspace,
                         size_t workspace_bytes, void* stream);
size_t selective_scan_backward_workspace_size(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G);
sr_status selective_scan_backward(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G,
                                  const void* u, int64_t ld_u, const void* delta, int64_t ld_delta,
                                  const void* z, int64_t ld_z, const void* Bm, int64_t ld_b,
                                  const void* Cm, int64_t ld_c, sr_dtype x_dtype, const float* A,
                                  const float* skip, const float* delta_bias, int delta_softplus,
                                  const float* h0, const int32_t* lengths, const void* dy,
                                  int64_t ld_dy, const float* dh_last, void* du, void* ddelta,
                                  void* dz, void* dB, void* dC, float* dA, float* dskip,
                                  float* ddelta_bias, float* dh0, void* workspace,
                                  size_t workspace_bytes, void* stream);
sr_status selective_step(int64_t B, int64_t D, int64_t N, int64_t G, const void* u, int64_t ld_u,
                         const void* delta, int64_t ld_delta, const void* z, int64_t ld_z,
                         const void* Bm, int64_t ld_b, const void* Cm, int64_t ld_c,
                         sr_dtype x_dtype, const float* A, const float* skip,
                         const float* delta_bias, int delta_softplus, const float* h_prev,
                         float* h_next, void* y, void* stream);

/*
 * Short causal convolution, a filter of K taps per channel:
 *
 *     c_t = bias + sum_{j<K} w_j x_{t-K+1+j},   y_t = silu(c_t)   (silu 0: c_t)
 *
 *   x, y        [B,T,D] in x_dtype, x as rows of ld_x.
 *   w, bias     [D,K] and [D] (or NULL: zeros) in w_dtype.
 *   state, last [B,K-1,D] in x_dtype: the K - 1 inputs in front of the first
 *               token, oldest first (NULL: zeros), and behind the sequence (NULL:
 *               not wanted).
 * Sums and activation are fp32; y is rounded once.  K from 1 to 8 (more:
 * SR_ERR_UNSUPPORTED).
 *
 * causal_conv_backward: dy and dlast (or NULL) are the gradients on y and last;
 * dx and dstate in x_dtype, dw and dbias in fp32; dbias and dstate may be NULL.
 *
 * causal_conv_step: one token, x and y [B,D]; state_next may be the same buffer as
 * state (NULL: zeros), else they must not overlap.
 */
sr_status causal_conv_forward(int64_t B, int64_t T, int64_t D, int64_t K, const void* x, int64_t ld_x,
                      sr_dtype x_dtype, const void* w, const void* bias, sr_dtype w_dtype, int silu,
                      const void* state, const int32_t* lengths, void* y, void* last, void* stream);
size_t causal_conv_backward_workspace_size(int64_t B, int64_t T, int64_t D, int64_t K,
                                           sr_dtype x_dtype);
sr_status causal_conv_backward(int64_t B, int64_t T, int64_t D, int64_t K, const void* x,
                               int64_t ld_x, sr_dtype x_dtype, const void* w, const void* bias,
                               sr_dtype w_dtype, int silu, const void* state,
                               const int32_t* lengths, const void* dy, int64_t ld_dy,
                               const void* dlast, void* dx, float* dw, float* dbias, void* dstate,
                               void* workspace, size_t workspace_bytes, void* stream);
sr_status causal_conv_step(int64_t B, int64_t D, int64_t K, const void* x, int64_t ld_x,
                           sr_dtype x_dtype, const void* w, const void* bias, sr_dtype w_dtype,
                           int silu, const void* state, void* state_next, void* y, void* stream);

/*
 * Root-mean-square norm of rows, with the residual's addition in front:
 *
 *     t = x + r   (rounded to r_dtype, stored as total),   y = t / sqrt(mean(t^2) + eps) w
 *
 *   x, y       [M,D] in x_dtype, x as rows of ld_x.
 *   r, total   [M,D] in r_dtype, or both NULL: t = x.  total may be the same
 *              buffer as r (rows of D then).
 *   w          [D] in w_dtype.
 * Sums are fp32; y is made of the sum as it is stored and rounded once.  D from 1 to
 * 16384 (more: SR_ERR_UNSUPPORTED).
 *
 * rms_norm_quantize: y as 8-bit codes with a scale per row, as quantize_rows makes
 * them, but of the fp32 values: q [M, quantized_row_bytes(D)] 16-byte aligned,
 * scale [M].
 *
 * rms_norm_backward: dy on y and dtotal (or NULL) on total give
 *     dx = (g - n mean(g n)) / rms + dtotal,   n = t / rms, g = dy w
 * in total_dtype, the gradient of x and of r, and dw = sum over rows of dy n in fp32.
 * total is the stored sum (x where there was no residual).
 */
sr_status rms_norm_forward(int64_t M, int64_t D, const void* x, int64_t ld_x, sr_dtype x_dtype,
                   const void* r, int64_t ld_r, sr_dtype r_dtype, const void* w, sr_dtype w_dtype,
                   float eps, void* total, void* y, void* stream);
sr_status rms_norm_quantize(int64_t M, int64_t D, const void* x, int64_t ld_x, sr_dtype x_dtype,
                            const void* r, int64_t ld_r, sr_dtype r_dtype, const void* w,
                            sr_dtype w_dtype, float eps, void* total, int8_t* q, float* scale,
                            void* stream);
size_t rms_norm_backward_workspace_size(int64_t M, int64_t D);
sr_status rms_norm_backward(int64_t M, int64_t D, const void* total, int64_t ld_total,
                            sr_dtype total_dtype, const void* w, sr_dtype w_dtype, float eps,
                            const void* dy, int64_t ld_dy, sr_dtype dy_dtype, const void* dtotal,
                            int64_t ld_dtotal, void* dx, float* dw, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Text of the last non-OK status returned on this thread ("" if none). */
const char* scanrnn_last_error(void);

/* Polls of a predecessor's unwritten look-back word after which a scan tile
 * gives up: it marks its workspace (see scanrnn_workspace_status) and
 * carries NaN for that channel instead of waiting longer (minGRU results are
 * NaN from there on; MinMax's min and max drop a NaN operand, so there only
 * the status shows it).  The default bound is never reached in normal
 * operation (predecessors are running, and publish within microseconds). */
#define SCANRNN_LOOKBACK_SPIN_LIMIT (1u << 20)

/* Lowers the bound above for scans launched afterwards by this process (all
 * threads; launches already enqueued keep theirs).  Meant for tests of the
 * timeout path: 0 gives up at the first unwritten word met.  polls above
 * SCANRNN_LOOKBACK_SPIN_LIMIT: SR_ERR_INVALID_ARGUMENT, nothing changed.
 * Pass SCANRNN_LOOKBACK_SPIN_LIMIT to restore the default. */
sr_status scanrnn_set_lookback_spin_limit(uint32_t polls);

/* Waits for `stream`, then reports what the scans that used `workspace` since
 * its last reset met: SR_ERR_LOOKBACK_TIMEOUT if one gave up waiting for a
 * predecessor chunk (a bounded wait that should never expire), else
 * SR_ERR_GATE_RANGE if a minGRU scan (forward, fused forward) met a gate
 * logit beyond the fp32 range of sigma (|k| above about 87.3; see the range
 * note at the top), else SR_OK. */
sr_status scanrnn_workspace_status(const void* workspace, void* stream);

/* Library version, "major.minor.patch". */
const char* scanrnn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SCANRNN_H */
