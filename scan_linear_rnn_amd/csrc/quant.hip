// Symmetric 8-bit codes with one scale per row (a token's activations) or per
// column (an output channel of a weight): what the 8-bit product reads.
//
//     s = max |x| / 127 (fp32),  q = rint(x / s) in [-127, 127]
//
// Both divisions are IEEE fp32 divisions, so the codes are a function of the
// inputs alone (no approximate reciprocal decides a tie).  A row of zeros
// has s = 0 and q = 0; a row with a NaN or an infinity has s = NaN and q = 0,
// so that whatever is computed from it is NaN.  The largest magnitude is
// taken on the bit patterns, which order like the values and put infinities
// and NaNs on top.
//
// Codes are stored as rows of quantized_width(K) bytes, zeros behind the K
// codes: the product then reads whole 128-byte lines, and the zeros add
// nothing to its integer sums.

#include "device_util.hpp"
#include "internal.hpp"

namespace sr {
namespace {

__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }

// The scale of a row whose largest magnitude has the bits `top`.
__device__ __forceinline__ float row_scale(uint32_t top) {
  return top < kF32InfBits ? __fdiv_rn(__uint_as_float(top), 127.0f) : __uint_as_float(0x7FC00000u);
}

// One code as a byte; `live` says that s is finite and above zero.
__device__ __forceinline__ uint32_t code(float x, float s, bool live) {
  const float q = rintf(__fdiv_rn(x, s));
  const int c = int(fminf(fmaxf(q, -127.0f), 127.0f));
  return live ? uint32_t(c) & 0xFFu : 0u;
}

// One row per workgroup, its elements read twice (the second time from the
// caches).
template <typename T>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T* x, int64_t ldx, int64_t K,
                                                            int64_t Kp, int8_t* q, float* scale) {
  __shared__ uint32_t s_top[4];
  const int64_t row = blockIdx.x;
  const T* src = x + row * ldx;
  uint32_t top = 0;
  for (int64_t k = threadIdx.x; k < K; k += 256) {
    const uint32_t b = abs_bits(load_f32(src + k));
    top = top > b ? top : b;
  }
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top;
  __syncthreads();
  top = s_top[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) top = top > s_top[w] ? top : s_top[w];
  const float s = row_scale(top);
  const bool live = s > 0.0f;
  if (threadIdx.x == 0) scale[row] = s;
  uint32_t* dst = reinterpret_cast<uint32_t*>(q + row * Kp);
  for (int64_t k = int64_t(threadIdx.x) * 4; k < Kp; k += 1024) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k + j < K) w |= code(load_f32(src + k + j), s, live) << (8 * j);
    dst[k / 4] = w;
  }
}

// Columns of W [K, N] (row-major) become rows of codes: a workgroup owns
// kColTile columns, finds their largest magnitudes over all K rows, then
// reads the rows again and writes four codes of a column at a time.
constexpr int kColTile = 16;

template <typename T>
__global__ __launch_bounds__(256) void quantize_columns_kernel(const T* W, int64_t ldw, int64_t K,
                                                               int64_t N, int64_t Kp, int8_t* q,
                                                               float* scale) {
  constexpr int kGroups = 256 / kColTile;  // row groups
  __shared__ uint32_t s_top[kGroups][kColTile];
  const int c = threadIdx.x % kColTile, r = threadIdx.x / kColTile;
  const int64_t n = int64_t(blockIdx.x) * kColTile + c;
  const bool on = n < N;
  uint32_t top = 0;
  if (on) {
    for (int64_t k = r; k < K; k += kGroups) {
      const uint32_t b = abs_bits(load_f32(W + k * ldw + n));
      top = top > b ? top : b;
    }
  }
  s_top[r][c] = top;
  __syncthreads();
#pragma unroll
  for (int g = 0; g < kGroups; ++g) top = top > s_top[g][c] ? top : s_top[g][c];
  if (!on) return;
  const float s = row_scale(top);
  const bool live = s > 0.0f;
  if (r == 0) scale[n] = s;
  uint32_t* dst = reinterpret_cast<uint32_t*>(q + n * Kp);
  for (int64_t k = int64_t(r) * 4; k < Kp; k += kGroups * 4) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k + j < K) w |= code(load_f32(W + (k + j) * ldw + n), s, live) << (8 * j);
    dst[k / 4] = w;
  }
}

sr_status launched(const char* what) {
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(SR_ERR_HIP, "%s launch: %s", what, hipGetErrorString(err));
  return SR_OK;
}

}  // namespace

sr_status launch_quantize_rows(int64_t M, int64_t K, const void* x, int64_t ldx, sr_dtype dtype,
                               int8_t* q, float* scale, hipStream_t stream, bool check_only) {
  if (M == 0) return SR_OK;
  if (M > kMaxBlocks256)
    return fail(SR_ERR_UNSUPPORTED, "%lld rows exceed one launch's grid", (long long)M);
  if (check_only) return SR_OK;
  const int64_t Kp = quantized_row_bytes(K);
  const dim3 grid{uint32_t(M)};
  if (dtype == SR_BF16)
    hipLaunchKernelGGL(quantize_rows_kernel<uint16_t>, grid, dim3(256), 0, stream,
                       static_cast<const uint16_t*>(x), ldx, K, Kp, q, scale);
  else
    hipLaunchKernelGGL(quantize_rows_kernel<float>, grid, dim3(256), 0, stream,
                       static_cast<const float*>(x), ldx, K, Kp, q, scale);
  return launched("row quantisation");
}

sr_status launch_quantize_columns(int64_t K, int64_t N, const void* W, int64_t ldw, sr_dtype dtype,
                                  int8_t* q, float* scale, hipStream_t stream) {
  if (N == 0) return SR_OK;
  const int64_t blocks = (N + kColTile - 1) / kColTile;
  if (blocks > kMaxBlocks256)
    return fail(SR_ERR_UNSUPPORTED, "%lld columns exceed one launch's grid", (long long)N);
  const int64_t Kp = quantized_row_bytes(K);
  const dim3 grid{uint32_t(blocks)};
  if (dtype == SR_BF16)
    hipLaunchKernelGGL(quantize_columns_kernel<uint16_t>, grid, dim3(256), 0, stream,
                       static_cast<const uint16_t*>(W), ldw, K, N, Kp, q, scale);
  else
    hipLaunchKernelGGL(quantize_columns_kernel<float>, grid, dim3(256), 0, stream,
                       static_cast<const float*>(W), ldw, K, N, Kp, q, scale);
  return launched("column quantisation");
}

}  // namespace sr
