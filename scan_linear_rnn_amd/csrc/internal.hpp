// Internal declarations shared by the host API and the kernel launchers.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "scanrnn.h"

namespace sr {

// Records a printf-style message as the calling thread's last error and
// returns `code`.
sr_status fail(sr_status code, const char* fmt, ...);

// Empties the calling thread's last-error text (each entry point starts so).
void clear_last_error();

// Polls of an unwritten look-back word after which a scan gives up (marks
// the workspace, publishes NaN): process-wide, SCANRNN_LOOKBACK_SPIN_LIMIT
// unless scanrnn_set_lookback_spin_limit lowered it.
uint32_t lookback_spin_limit();

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

constexpr size_t kAlign = 256;

// ---------------------------------------------------------------- scan engine
//
// The workspace of one scan: a 256-byte header (ticket counter, status word)
// followed by one 64-bit state word per (chunk along T, batch row, channel).

struct ScanGeometry {
  int V;             // channels per lane
  int N;             // time steps per lane
  int W;             // waves per workgroup (stacked along T)
  int64_t Dc;        // channels per workgroup = 64 * V
  int64_t Tc;        // time steps per workgroup = W * N
  int64_t n_dtiles;  // ceil(D / Dc)
  int64_t n_tchunks; // ceil(T / Tc)
};

// Largest workspace any geometry needs for a [B,T,D] scan.
size_t scan_workspace_bytes(int64_t B, int64_t T, int64_t D);

enum class ScanOp { kMinGRU, kMinMax };

struct ScanRequest {
  ScanOp op;
  sr_dtype in_dtype;   // k,p (minGRU) or r,s (MinMax, fp32 only)
  int64_t B, T, D;
  const void* in0;     // k or r
  const void* in1;     // p or s
  int64_t ld_in;       // row stride of in0/in1, elements
  const float* init;   // h0 / x0 [B,D] or nullptr (zero state)
  float* out;          // [B,T,D] contiguous
  float* last;         // [B,D] or nullptr
  void* workspace;
  hipStream_t stream;
  // Time decay of the carried state (minGRU only; none when decay_rate is null).
  const float* decay_rate = nullptr;  // [D]
  const float* delta_t = nullptr;     // [B,T], contiguous
  int log1p_delta = 0;
  uint32_t* saturated = nullptr;      // device flag, OR-ed with 1 on saturation
  // Run every check the launch makes, then return without enqueuing
  // anything (so that a call of several launches can check them all first).
  bool check_only = false;
};

sr_status launch_scan(const ScanRequest& rq);

// Chooses the geometry a request will use (exposed for sizing and tests).
ScanGeometry choose_geometry(const ScanRequest& rq);

// Fused input projection + scan (fused.hip): h = scan(x W_in), the [k|p]
// tile never leaving the workgroup.  Used for large enough problems (see
// fused_forward_applies); its workspace is the look-back words of its own
// 256-step tiles.
struct FusedRequest {
  int64_t B, T, D_in, D_h;
  const float* x;      // [B,T,D_in]
  const float* W_in;   // [D_in, 2*D_h]
  const float* h0;     // [B,D_h] or nullptr
  float* h;            // [B,T,D_h]
  float* h_last;       // [B,D_h] or nullptr
  void* workspace;
  hipStream_t stream;
  const float* decay_rate = nullptr;  // time decay, as in ScanRequest
  const float* delta_t = nullptr;
  int log1p_delta = 0;
  uint32_t* saturated = nullptr;
  bool check_only = false;  // as in ScanRequest
};

bool fused_forward_applies(int64_t B, int64_t T, int64_t D_h);
size_t fused_workspace_bytes(int64_t B, int64_t T, int64_t D_h);
sr_status launch_fused_forward(const FusedRequest& rq);

// Backward pass of a scan (reverse time, same engine).
struct BackwardRequest {
  ScanOp op;
  sr_dtype in_dtype;    // k,p (minGRU); r,s are fp32
  int64_t B, T, D;
  const void* in0;      // k or r
  const void* in1;      // p or s
  int64_t ld_in;
  const float* fwd;     // forward outputs [B,T,D] (h_t or x_{t+1})
  const float* fwd0;    // forward initial state [B,D] (null = zero; required for MinMax)
  const float* grad;    // upstream gradient [B,T,D]
  const float* grad_last;  // gradient on the returned final state [B,D] or null
  float* d0;            // dk or dr [B,T,D]
  float* d1;            // dp or ds [B,T,D]
  float* dinit;         // dh0 or dx0 [B,D] or null
  // Time decay of the carried state (minGRU only; none when decay_rate is null).
  const float* decay_rate;  // [D]
  const float* delta_t;     // [B,T]
  int log1p_delta;
  void* workspace;
  hipStream_t stream;
};

sr_status launch_scan_backward(const BackwardRequest& rq);
size_t scan_backward_workspace_bytes(int64_t B, int64_t T, int64_t D);

// ---------------------------------------------------------------- GEMM
//
// C[M,N] = A[M,K] * B[K,N], fp32, row-major with leading dimensions.  Small
// problems split K across workgroups; `ws` must then hold
// gemm_workspace_bytes(M, N, K, false) bytes (it may be null when that is 0).
// With check_only, every check is made and nothing is enqueued.
sr_status launch_gemm_f32(int64_t M, int64_t N, int64_t K,
                          const float* A, int64_t lda,
                          const float* Bm, int64_t ldb,
                          float* C, int64_t ldc, float* ws, hipStream_t stream,
                          bool check_only = false);

// Time decay of the carried state in the step (see mingru_step_decayed).
struct StepDecay {
  const float* rate;     // [D_h]
  const float* gap;      // [Bsz]
  int log1p_gap;
  uint32_t* saturated;   // or null
};

// Step kernel: h_next = (1 - z) gamma h_prev + z g(p) with [k|p] = x_t W_in
// (gamma = 1 without decay), computed as one GEMM whose epilogue applies the
// update.  `ws`: as above with gemm_workspace_bytes(Bsz, 2*D_h, D_in, true).
sr_status launch_step_in(int64_t Bsz, int64_t D_in, int64_t D_h,
                         const float* x_t, const float* W_in,
                         const float* h_prev, float* h_next, float* ws, hipStream_t stream,
                         const StepDecay* decay = nullptr, bool check_only = false);

// Number of K slices a GEMM of this shape uses, and the workspace they need.
int gemm_splits(int64_t M, int64_t N, int64_t K, bool step);
size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, bool step);

// ------------------------------------------------- 8-bit codes and products

// Rows of codes are padded with zeros to a multiple of this many bytes.
constexpr int64_t kI8Align = 128;
inline int64_t quantized_row_bytes(int64_t K) { return (K + kI8Align - 1) / kI8Align * kI8Align; }
// Deepest product whose sums fit 32 bits: 127^2 * K < 2^31.
constexpr int64_t kMaxI8Depth = 131072;
// Workgroups of 256 threads in one launch (a 1-D grid has at most 2^32 work-items).
constexpr int64_t kMaxBlocks256 = int64_t(0xFFFFFFFF) / 256;

// Codes q [M, quantized_row_bytes(K)] and scales [M] of x (rows of ldx elements).
sr_status launch_quantize_rows(int64_t M, int64_t K, const void* x, int64_t ldx, sr_dtype dtype,
                               int8_t* q, float* scale, hipStream_t stream, bool check_only = false);

// Codes q [N, quantized_row_bytes(K)] and scales [N] of the columns of W [K, N].
sr_status launch_quantize_columns(int64_t K, int64_t N, const void* W, int64_t ldw, sr_dtype dtype,
                                  int8_t* q, float* scale, hipStream_t stream);

// Rows that a product quantises itself, instead of codes and scales in A and
// a_scale: at most a few, contiguous (see tokens_apply).
struct Tokens {
  const void* x;  // [M, K]
  int64_t K;
  sr_dtype dtype;
};
bool tokens_apply(int64_t M, int64_t K, const void* x, sr_dtype dtype);

// C[M,N] = (A B^T) a_scale b_scale over codes A [M,K], B [N,K] (K a multiple
// of kI8Align, rows 16-byte aligned).
sr_status launch_gemm_i8(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda,
                         const float* a_scale, const int8_t* B, int64_t ldb, const float* b_scale,
                         void* C, int64_t ldc, sr_dtype c_dtype, hipStream_t stream,
                         bool check_only = false, const Tokens* tokens = nullptr);

// The step on codes: [k|p] = the product of x [Bsz,K] and W_in [2 D_h, K],
// h_next as in launch_step_in.
sr_status launch_step_i8(int64_t Bsz, int64_t K, int64_t D_h, const int8_t* x, const float* x_scale,
                         const int8_t* W_in, const float* w_scale, const float* h_prev,
                         float* h_next, hipStream_t stream, const StepDecay* decay,
                         bool check_only = false, const Tokens* tokens = nullptr);

// ---------------------------------------------------------------- AdamW

// Elements of a tensor that share a scale of the 8-bit states; also what a
// tensor's span in the state buffers is rounded up to.
constexpr int64_t kStateBlock = 256;
inline int64_t adamw_span(int64_t n) { return (n + kStateBlock - 1) / kStateBlock * kStateBlock; }

struct AdamWRequest {
  int64_t n_tensors;
  const sr_adamw_tensor* tensors;  // host memory
  void* m;
  void* v;
  float* m_scale;  // null: fp32 states
  float* v_scale;
  int64_t step;          // of every tensor, where steps is null
  const int64_t* steps;  // host memory: of each tensor
  double lr, beta1, beta2, eps, weight_decay;
  const float* grad_scale;
  hipStream_t stream;
};

sr_status launch_adamw(const AdamWRequest& rq);

// ------------------------------------------------- selective state space scan

constexpr int kSelectiveTile = 16;        // tokens a workgroup handles between barriers
constexpr int kSelectiveStates = 64;      // most states per channel
constexpr int64_t kSelectiveRow = int64_t(1) << 25;  // furthest that rows of several tokens may be apart
constexpr int64_t kSelectiveMinTokens = 128;  // tokens of the shortest sequence that is cut

// How a call is cut: 64 channels of a group per workgroup, the tokens in chunks.
struct SelectivePlan {
  int64_t tiles_per_group;
  int64_t chunks, chunk_len;  // chunk_len a multiple of kSelectiveTile where there are several
};
SelectivePlan selective_plan(int64_t B, int64_t T, int64_t D, int64_t G);
SelectivePlan selective_backward_plan(int64_t B, int64_t T, int64_t D, int64_t G);

// The operands of the calls (scanrnn.h) and the areas of their workspaces.
struct SelectiveRequest {
  sr_dtype dtype;
  int64_t B, T, D;
  int N, G;
  const void *u, *delta, *z;  // z may be null
  int64_t ld_u, ld_delta, ld_z;
  const float* A;
  const void *Bm, *Cm;
  int64_t ld_b, ld_c;
  const float *skip, *bias;  // may be null
  int softplus;
  const float* h0;  // may be null; the step's h_prev
  const int32_t* lengths;
  void* y;
  float* h_last;  // may be null; the step's h_next
  int tiles_per_group;
  int chunks;
  int64_t chunk_len;
  float* ends;   // [chunks][B][N][D]
  float* steps;  // [chunks][B][D]
  float* marks;  // [T / 16][B][N + 1][D], or null
  hipStream_t stream;
  // The backward pass.
  const void* dy;
  int64_t ld_dy;
  const float* dh_last;  // may be null
  void *du, *ddelta, *dz, *dB, *dC;
  float *dA, *dskip, *dbias, *dh0;  // dskip, dbias, dh0 may be null
  float* gends;   // [chunks][B][N][D]
  float* parts;   // dB and dC of each 64 channels: [tile][B][T][2][states rounded up]
  float* aparts;  // dA, dskip and dbias of each sequence and chunk: [B][chunks][N + 2][D]
};

sr_status launch_selective_scan(const SelectiveRequest& rq);
sr_status launch_selective_states(const SelectiveRequest& rq);
sr_status launch_selective_carry(const SelectiveRequest& rq, const float* init, float* last, bool reverse);
sr_status launch_selective_backward(const SelectiveRequest& rq);
int64_t selective_step_blocks(int64_t B, int64_t D, int64_t N);  // workgroups of 256
sr_status launch_selective_step(const SelectiveRequest& rq);
// Threads of its largest workgroup: four waves or eight.
inline int selective_threads(int64_t N, bool backward) { return N <= (backward ? 8 : 16) ? 256 : 512; }
// States of one row of `parts`: N rounded up to what the workgroup's waves hold.
inline int64_t selective_padded(int64_t N) { return N <= 4 ? 4 : N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }

// ------------------------------------------------- short causal convolution

constexpr int kConvTaps = 8;  // most taps per channel

struct ConvPlan {
  int64_t run_len, runs;  // tokens of a thread, and runs per sequence
};
ConvPlan conv_plan(int64_t B, int64_t T, int64_t D, sr_dtype dtype, bool backward);

struct ConvRequest {
  sr_dtype dtype, w_dtype;
  int64_t B, T, D;
  int K;
  const void* x;
  int64_t ld_x;
  const void *w, *bias;  // bias may be null
  int silu;
  const void* state;  // [B][K - 1][D] or null
  const int32_t* lengths;
  void *y, *last;  // last may be null
  int64_t run_len, runs;
  hipStream_t stream;
  // The backward pass.
  const void* dy;
  int64_t ld_dy;
  const void* dlast;  // may be null
  void *dx, *dstate;  // dstate may be null
  float *dw, *dbias;  // dbias may be null
  float* parts;       // [B][runs][K + 1][D]
};

// Threads of their launches, in workgroups of 256.
int64_t conv_threads(const ConvRequest& rq);
int64_t conv_backward_threads(const ConvRequest& rq);
int64_t conv_step_threads(const ConvRequest& rq);
sr_status launch_conv(const ConvRequest& rq);
sr_status launch_conv_backward(const ConvRequest& rq);
sr_status launch_conv_step(const ConvRequest& rq);

// ------------------------------------------------- root-mean-square norm

constexpr int64_t kNormWidth = 16384;  // longest row

struct NormRequest {
  sr_dtype dtype, r_dtype, w_dtype;
  int64_t M, D;
  const void *x, *r;  // r may be null
  int64_t ld_x, ld_r;
  const void* w;
  float eps;
  void *total, *y;
  int8_t* q;  // null: y
  float* scale;
  int64_t ld_q;
  hipStream_t stream;
  // The backward pass.
  const void *t, *dy, *dt;  // dt may be null
  int64_t ld_t, ld_dy, ld_dt;
  void* dx;
  float* dw;
  float* parts;  // [norm_backward_blocks][D]
};

int64_t norm_backward_blocks(int64_t M, int64_t D);
sr_status launch_norm(const NormRequest& rq);
sr_status launch_norm_backward(const NormRequest& rq);

// One MinMax step over n channels (x_next may alias x_prev).
sr_status launch_minmax_step(const float* r, const float* s, const float* x_prev, float* x_next,
                             int64_t n, hipStream_t stream);

// Copies n floats (src may be null: writes zeros).
sr_status launch_copy_or_zero(float* dst, const float* src, int64_t n, hipStream_t stream);

}  // namespace sr
