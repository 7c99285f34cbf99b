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

#include "internal.hpp"
#include "quant.hpp"

namespace sr {
namespace {

__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }

// WPR waves per row, NV 16-byte chunks per lane: the row is read once and
// stays in registers.  Loads go through a descriptor that ends with the row,
// so chunks past its end are zeros and become the padding.  Bound by the
// bytes of a large x (131072 x 2048 fp32: see the launch), by latency for a
// few rows, which is why those take four waves each.
template <typename T, int WPR, int NV>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T* x, int64_t ldx, int64_t M, int K,
                                                            int Kp, int8_t* q, float* scale) {
  using C = Chunk<T>;
  __shared__ uint32_t s_top[4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t row = int64_t(blockIdx.x) * (4 / WPR) + wave / WPR;
  if (row >= M) return;  // (WPR == 4: never)
  const int c0 = wave % WPR * 64 + lane;
  // bf16 rows of odd length end within a dword, whose other half is masked.
  const int bytes = (K * int(sizeof(T)) + 3) & ~3;
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(x + row * ldx), 0, bytes, 0x00020000);
  u32x4 w[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    w[j] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, (c0 + j * 64 * WPR) * 16, 0, 2);
  if (sizeof(T) == 2 && (K & 1)) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int d = 0; d < 4; ++d)
        if ((c0 + j * 64 * WPR) * 8 + d * 2 + 1 == K) w[j][d] &= 0xFFFFu;
  }
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t t = C::top(w[j]);
    top = top > t ? top : t;
  }
  top = wave_max(top);
  if constexpr (WPR == 4) {
    if (lane == 0) s_top[wave] = top;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < 4; ++v) top = top > s_top[v] ? top : s_top[v];
  }
  const float s = row_scale(top);
  if (c0 == 0) scale[row] = s;
  int8_t* dst = q + row * int64_t(Kp);
  const bool plain = divides_plainly(s);
  const float r = plain ? __fdiv_rn(1.0f, s) : 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int k = (c0 + j * 64 * WPR) * C::kSize;
    uint32_t codes[C::kSize / 4];
    C::codes(w[j], s, r, plain, codes);
    if (k < Kp) {
      if constexpr (C::kSize == 8)
        __builtin_nontemporal_store(u32x2{codes[0], codes[1]}, reinterpret_cast<u32x2*>(dst + k));
      else
        __builtin_nontemporal_store(codes[0], reinterpret_cast<uint32_t*>(dst + k));
    }
  }
}

// Rows too long for registers, or of bf16 at odd elements: one per workgroup,
// read twice (the second time from the caches).
template <typename T>
__global__ __launch_bounds__(256) void quantize_any_rows_kernel(const T* x, int64_t ldx, int64_t K,
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
#pragma unroll
  for (int w = 0; w < 4; ++w) top = top > s_top[w] ? top : s_top[w];
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

// Columns of W [K, N] (row-major) become rows of codes.  A workgroup of 1024
// threads owns 64 bytes of columns, four threads to a row; a thread holds four
// consecutive rows of a pass of 1024, so that it writes four codes of a
// column as one dword, and all of W is read once.  Neighbouring workgroups
// share the other half of each line, so each XCD takes a contiguous range.
template <typename T, int NP>
__global__ __launch_bounds__(1024) void quantize_columns_kernel(const T* W, int64_t ldw, int K, int64_t N,
                                                                int Kp, int8_t* q, float* scale) {
  using C = Chunk<T>;
  constexpr int V = C::kSize, kCols = 4 * V;
  __shared__ uint32_t s_top[16][kCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t per = gridDim.x / 8;
  const uint32_t tile = blockIdx.x < per * 8 ? (blockIdx.x % 8) * per + blockIdx.x / 8 : blockIdx.x;
  const int64_t n0 = int64_t(tile) * kCols;
  const int c = (threadIdx.x & 3) * V, g = threadIdx.x >> 2;
  // Rows past K fall behind the descriptor's end and read as zeros; columns
  // past N read the next row's and are not stored.
  const int64_t elements = int64_t(K - 1) * ldw + (N - n0);
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<T*>(W + n0), 0, int(uint32_t((elements * int64_t(sizeof(T)) + 3) & ~int64_t(3))), 0x00020000);
  u32x4 w[NP][4];
  const uint32_t row_bytes = uint32_t(ldw * int64_t(sizeof(T)));
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = p * 1024 + 4 * g + i;
      const uint32_t off = uint32_t(k) * row_bytes + uint32_t(c * int(sizeof(T)));
      w[p][i] = u32x4{};
      if (k < K) w[p][i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, int(off), 0, 0);
    }
  uint32_t top[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    top[e] = 0;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = abs_bits(C::get(w[p][i], e));
        top[e] = top[e] > b ? top[e] : b;
      }
#pragma unroll
    for (int d = 4; d < 64; d <<= 1) {
      const uint32_t o = __shfl_xor(top[e], d);
      top[e] = top[e] > o ? top[e] : o;
    }
  }
  if (lane < 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) s_top[wave][c + e] = top[e];
  }
  __syncthreads();
  if (threadIdx.x < kCols) {
    uint32_t t = 0;
#pragma unroll
    for (int v = 0; v < 16; ++v) t = t > s_top[v][threadIdx.x] ? t : s_top[v][threadIdx.x];
    s_top[0][threadIdx.x] = t;  // (only this thread reads the column)
    if (n0 + threadIdx.x < N) scale[n0 + threadIdx.x] = row_scale(t);
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if (n0 + c + e >= N) break;
    const float s = row_scale(s_top[0][c + e]);
    const bool live = s > 0.0f, plain = divides_plainly(s);
    const float r = plain ? __fdiv_rn(1.0f, s) : 0.0f;
    int8_t* dst = q + (n0 + c + e) * int64_t(Kp);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int k = p * 1024 + 4 * g;
      if (k >= Kp) break;
      uint32_t v = 0;
      if (plain) {
#pragma unroll
        for (int i = 3; i >= 0; --i)
          v = (v << 8) | (uint32_t(int(rintf(divided(C::get(w[p][i], e), s, r)))) & 0xFFu);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v |= code(C::get(w[p][i], e), s, live) << (8 * i);
      }
      *reinterpret_cast<uint32_t*>(dst + k) = v;
    }
  }
}

// Columns that the kernel above does not take (K beyond its registers, bf16
// at odd elements, 4 GiB and more): a workgroup owns kColTile columns, finds
// their largest magnitudes over all K rows, then reads the rows again.
constexpr int kColTile = 16;

template <typename T>
__global__ __launch_bounds__(256) void quantize_any_columns_kernel(const T* W, int64_t ldw, int64_t K,
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

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <typename T, int WPR>
void launch_rows(int nv, int64_t M, int K, int Kp, const T* x, int64_t ldx, int8_t* q, float* scale,
                 hipStream_t stream) {
  const dim3 grid{uint32_t((M + 4 / WPR - 1) / (4 / WPR))}, block{256};
#define SR_ROWS(NV)                                                                                       \
  hipLaunchKernelGGL((quantize_rows_kernel<T, WPR, NV>), grid, block, 0, stream, x, ldx, M, K, Kp, q, scale)
  if (nv <= 1) SR_ROWS(1);
  else if (nv <= 2) SR_ROWS(2);
  else if (nv <= 4) SR_ROWS(4);
  else if (nv <= 8) SR_ROWS(8);
  else SR_ROWS(16);
#undef SR_ROWS
}

// Chunks per lane that the kernels for whole rows go up to.
constexpr int kMaxChunks = 16;
// Fewer rows than this take four waves each: a wave per row would leave SIMDs idle.
constexpr int64_t kFewRows = 1024;

template <typename T>
void launch_rows(int64_t M, int64_t K, const T* x, int64_t ldx, int8_t* q, float* scale,
                 hipStream_t stream) {
  const int64_t Kp = quantized_row_bytes(K);
  const int64_t chunks = (Kp * int64_t(sizeof(T)) + 15) / 16;  // Kp: the padding is written too
  const bool dwords = sizeof(T) == 4 || (ldx % 2 == 0 && aligned(x, 4)) || (M == 1 && aligned(x, 4));
  if (K == 0 || !dwords || chunks > 4 * 64 * kMaxChunks)
    hipLaunchKernelGGL(quantize_any_rows_kernel<T>, dim3(uint32_t(M)), dim3(256), 0, stream, x, ldx, K, Kp, q,
                       scale);
  else if (M < kFewRows || chunks > 64 * kMaxChunks)
    launch_rows<T, 4>(int((chunks + 255) / 256), M, int(K), int(Kp), x, ldx, q, scale, stream);
  else
    launch_rows<T, 1>(int((chunks + 63) / 64), M, int(K), int(Kp), x, ldx, q, scale, stream);
}

}  // namespace

sr_status launch_quantize_rows(int64_t M, int64_t K, const void* x, int64_t ldx, sr_dtype dtype,
                               int8_t* q, float* scale, hipStream_t stream, bool check_only) {
  if (M == 0) return SR_OK;
  if (M > kMaxBlocks256)
    return fail(SR_ERR_UNSUPPORTED, "%lld rows exceed one launch's grid", (long long)M);
  if (check_only) return SR_OK;
  if (dtype == SR_BF16)
    launch_rows(M, K, static_cast<const uint16_t*>(x), ldx, q, scale, stream);
  else
    launch_rows(M, K, static_cast<const float*>(x), ldx, q, scale, stream);
  return launched("row quantisation");
}

namespace {

template <typename T>
void launch_columns(int64_t K, int64_t N, const T* W, int64_t ldw, int8_t* q, float* scale,
                    hipStream_t stream) {
  const int64_t Kp = quantized_row_bytes(K);
  const bool dwords = sizeof(T) == 4 || ((ldw % 2 == 0 || K == 1) && aligned(W, 4));
  if (K == 0 || K > 4096 || !dwords || K * ldw * int64_t(sizeof(T)) > int64_t(0xFFFFFFFF) - 256) {
    hipLaunchKernelGGL(quantize_any_columns_kernel<T>, dim3(uint32_t((N + kColTile - 1) / kColTile)), dim3(256), 0,
                       stream, W, ldw, K, N, Kp, q, scale);
    return;
  }
  constexpr int kCols = 4 * Chunk<T>::kSize;
  const dim3 grid{uint32_t((N + kCols - 1) / kCols)}, block{1024};
  if (K <= 1024)
    hipLaunchKernelGGL((quantize_columns_kernel<T, 1>), grid, block, 0, stream, W, ldw, int(K), N, int(Kp), q, scale);
  else if (K <= 2048)
    hipLaunchKernelGGL((quantize_columns_kernel<T, 2>), grid, block, 0, stream, W, ldw, int(K), N, int(Kp), q, scale);
  else
    hipLaunchKernelGGL((quantize_columns_kernel<T, 4>), grid, block, 0, stream, W, ldw, int(K), N, int(Kp), q, scale);
}

}  // namespace

sr_status launch_quantize_columns(int64_t K, int64_t N, const void* W, int64_t ldw, sr_dtype dtype,
                                  int8_t* q, float* scale, hipStream_t stream) {
  if (N == 0) return SR_OK;
  if (N > kMaxBlocks256)
    return fail(SR_ERR_UNSUPPORTED, "%lld columns exceed one launch's grid", (long long)N);
  if (dtype == SR_BF16)
    launch_columns(K, N, static_cast<const uint16_t*>(W), ldw, q, scale, stream);
  else
    launch_columns(K, N, static_cast<const float*>(W), ldw, q, scale, stream);
  return launched("column quantisation");
}

}  // namespace sr
