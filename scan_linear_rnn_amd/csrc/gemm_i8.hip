// 8-bit integer product with a scale per row of either operand, and the
// single-token minGRU step on it:
//
//     c[m, n] = (sum_k a[m, k] b[n, k]) (s_m t_n)
//
// The sum is exact in 32-bit integers (|a|, |b| <= 127 and K <= kMaxI8Depth
// keep it below 2^31), so neither the order of the sum nor the tiling
// changes a result; it is rounded once to fp32, multiplied by the product of
// the scales, and rounded once more if the output is bf16.
//
// Operand layout of v_mfma_i32_16x16x64_i8 (one 16 x 16 x 64 product per
// wave): lane l supplies 16 consecutive k of row l % 16, k from 16 (l / 16);
// accumulator r of lane l is D[4 (l / 16) + r][l % 16].  The weights go in
// as the left operand, so that a lane ends with four consecutive output
// columns of one row: 16-byte stores, and in the step four channels whose
// states are one 16-byte load and store.

#include "device_util.hpp"
#include "internal.hpp"
#include "step_gate.hpp"

namespace sr {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct I8Params {
  int64_t M, N, K;  // N: output columns (step: 2 D_h); K: stored width, a multiple of kI8Align
  const int8_t* A;
  int64_t lda;
  const float* a_scale;  // [M]
  const int8_t* B;
  int64_t ldb;
  const float* b_scale;  // [N]
  void* C;               // [M, N], rows of ldc elements
  int64_t ldc;
  int vec;               // rows of C (step: of the states) allow 4-element accesses
  // step: k and p are columns d and D_h + d
  int64_t D_h;
  const float* h_prev;
  float* h_next;
  const float* rate;
  const float* gap;
  int log1p_gap;
  uint32_t* saturated;
};

enum Out { kF32 = 0, kBF16 = 1, kStep = 2 };

__device__ __forceinline__ float scaled(int acc, float s, float t) { return float(acc) * (s * t); }

// Stores four consecutive columns of row m, from column n.
template <int OUT>
__device__ __forceinline__ void store4(const I8Params& P, int64_t m, int64_t n, f32x4 v) {
  if (m >= P.M) return;
  if (OUT == kF32) {
    float* dst = static_cast<float*>(P.C) + m * P.ldc + n;
    if (P.vec && n + 4 <= P.N) {
      *reinterpret_cast<f32x4*>(dst) = v;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < P.N) dst[j] = v[j];
    }
  } else {
    uint16_t* dst = static_cast<uint16_t*>(P.C) + m * P.ldc + n;
    if (P.vec && n + 4 <= P.N) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(bf16_bits(v[0]) | (bf16_bits(v[1]) << 16),
                                                  bf16_bits(v[2]) | (bf16_bits(v[3]) << 16));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < P.N) dst[j] = uint16_t(bf16_bits(v[j]));
    }
  }
}

// Scales of four consecutive columns (zeros past `end`).
__device__ __forceinline__ f32x4 scales4(const float* t, int64_t n, int64_t end) {
  f32x4 s;
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j] = n + j < end ? t[n + j] : 0.0f;
  return s;
}

// Epilogue of one 16 x 16 block pair of the step: four channels d .. d + 3 of
// row m, from their k and p sums.
__device__ __forceinline__ void step4(const I8Params& P, int64_t m, int64_t d, i32x4 k, i32x4 p) {
  if (m >= P.M) return;
  const float s = P.a_scale[m];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (d + j < P.D_h) {
      const float kk = scaled(k[j], s, P.b_scale[d + j]);
      const float pp = scaled(p[j], s, P.b_scale[P.D_h + d + j]);
      P.h_next[m * P.D_h + d + j] = step_value(kk, pp, carried_state(P, m, d + j));
    }
  }
}

// A workgroup of four waves computes 64 rows x 64 columns (step: 64 rows x
// 32 channels, k and p of each), a wave 32 x 32 of them as 2 x 2 products;
// operands go from global memory straight to registers.
template <int OUT>
__global__ __launch_bounds__(256) void i8_direct_kernel(const I8Params P) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lk = lane >> 4;
  const int64_t cols = OUT == kStep ? P.D_h : P.N;
  const int64_t tiles_m = (P.M + 63) / 64;
  const int64_t m0 = int64_t(blockIdx.x % uint32_t(tiles_m)) * 64 + (wave & 1) * 32;
  constexpr int kSpan = OUT == kStep ? 32 : 64;  // columns (channels) per workgroup
  const int64_t n0 = int64_t(blockIdx.x / uint32_t(tiles_m)) * kSpan + (wave >> 1) * (kSpan / 2);
  // Rows past the end repeat the last one: their results are not stored.
  const int8_t* pa[2];
  const int8_t* pb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + i * 16 + lr;
    pa[i] = P.A + (m < P.M ? m : P.M - 1) * P.lda + lk * 16;
    int64_t n = n0 + lr + (OUT == kStep ? 0 : i * 16);
    n = n < cols ? n : cols - 1;
    pb[i] = P.B + (n + (OUT == kStep ? i * P.D_h : 0)) * P.ldb + lk * 16;
  }
  i32x4 acc[2][2] = {};
  for (int64_t k = 0; k < P.K; k += 64) {
    i32x4 a[2], b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = *reinterpret_cast<const i32x4*>(pa[i] + k);
      b[i] = *reinterpret_cast<const i32x4*>(pb[i] + k);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[j], a[i], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + i * 16 + lr;
    if constexpr (OUT == kStep) {
      step4(P, m, n0 + 4 * lk, acc[i][0], acc[i][1]);
    } else {
      const float s = m < P.M ? P.a_scale[m] : 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t n = n0 + j * 16 + 4 * lk;
        const f32x4 t = scales4(P.b_scale, n, P.N);
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = scaled(acc[i][j][r], s, t[r]);
        store4<OUT>(P, m, n, v);
      }
    }
  }
}

sr_status launch(int out, const I8Params& P, hipStream_t stream, bool check_only) {
  const int64_t cols = out == kStep ? P.D_h : P.N;
  const int64_t span = out == kStep ? 32 : 64;
  const int64_t tiles_m = (P.M + 63) / 64, tiles_n = (cols + span - 1) / span;
  if (tiles_m > kMaxBlocks256 || tiles_n > kMaxBlocks256 || tiles_m * tiles_n > kMaxBlocks256)
    return fail(SR_ERR_UNSUPPORTED, "8-bit product of %lld x %lld tiles too large for one launch",
                (long long)tiles_m, (long long)tiles_n);
  if (check_only) return SR_OK;
  const dim3 grid{uint32_t(tiles_m * tiles_n)};
  if (out == kStep)
    hipLaunchKernelGGL(i8_direct_kernel<kStep>, grid, dim3(256), 0, stream, P);
  else if (out == kBF16)
    hipLaunchKernelGGL(i8_direct_kernel<kBF16>, grid, dim3(256), 0, stream, P);
  else
    hipLaunchKernelGGL(i8_direct_kernel<kF32>, grid, dim3(256), 0, stream, P);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(SR_ERR_HIP, "8-bit product launch: %s", hipGetErrorString(err));
  return SR_OK;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

sr_status launch_gemm_i8(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda,
                         const float* a_scale, const int8_t* B, int64_t ldb, const float* b_scale,
                         void* C, int64_t ldc, sr_dtype c_dtype, hipStream_t stream,
                         bool check_only) {
  if (M == 0 || N == 0) return SR_OK;
  I8Params P{};
  P.M = M; P.N = N; P.K = K;
  P.A = A; P.lda = lda; P.a_scale = a_scale;
  P.B = B; P.ldb = ldb; P.b_scale = b_scale;
  P.C = C; P.ldc = ldc;
  P.vec = ldc % 4 == 0 && aligned(C, c_dtype == SR_BF16 ? 8 : 16);
  return launch(c_dtype == SR_BF16 ? kBF16 : kF32, P, stream, check_only);
}

sr_status launch_step_i8(int64_t Bsz, int64_t K, int64_t D_h, const int8_t* x, const float* x_scale,
                         const int8_t* W_in, const float* w_scale, const float* h_prev,
                         float* h_next, hipStream_t stream, const StepDecay* decay,
                         bool check_only) {
  if (Bsz == 0 || D_h == 0) return SR_OK;
  I8Params P{};
  P.M = Bsz; P.N = 2 * D_h; P.K = K;
  P.A = x; P.lda = K; P.a_scale = x_scale;
  P.B = W_in; P.ldb = K; P.b_scale = w_scale;
  P.D_h = D_h; P.h_prev = h_prev; P.h_next = h_next;
  P.vec = D_h % 4 == 0 && aligned(h_prev, 16) && aligned(h_next, 16);
  if (decay != nullptr) {
    P.rate = decay->rate;
    P.gap = decay->gap;
    P.log1p_gap = decay->log1p_gap;
    P.saturated = decay->saturated;
  }
  return launch(kStep, P, stream, check_only);
}

}  // namespace sr
