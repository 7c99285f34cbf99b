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
// Codes are stored as rows of quantized_row_bytes(K) bytes, zeros behind the K
// codes: the product then reads whole 128-byte lines, and the zeros add
// nothing to its integer sums.

#include "internal.hpp"
#include "quant.hpp"

namespace sr {
namespace {

__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }

// The elements of w from element n on (n < the chunk's size), zeros behind them.
template <typename T>
__device__ __forceinline__ u32x4 from_element(u32x4 w, int n) {
  const int dwords = n * int(sizeof(T)) / 4;
  if (dwords & 2) w = u32x4{w[2], w[3], 0, 0};
  if (dwords & 1) w = u32x4{w[1], w[2], w[3], 0};
  if (sizeof(T) == 2 && (n & 1))
    w = u32x4{w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, w[3] >> 16};
  return w;
}

// 16 bytes from any element: global loads take any even address.
template <typename T>
__device__ __forceinline__ u32x4 load16(const T* p) {
  u32x4 w;
  __builtin_memcpy(&w, __builtin_assume_aligned(p, sizeof(T)), 16);
  return w;
}

// A chunk's codes: four or eight bytes.
__device__ __forceinline__ void store_codes(const uint32_t (&c)[1], int8_t* dst) {
  __builtin_nontemporal_store(c[0], reinterpret_cast<uint32_t*>(dst));
}
__device__ __forceinline__ void store_codes(const uint32_t (&c)[2], int8_t* dst) {
  __builtin_nontemporal_store(u32x2{c[0], c[1]}, reinterpret_cast<u32x2*>(dst));
}

// WPR waves per row, NV 16-byte chunks per lane: the row is read once and
// stays in registers; chunks past its end are zeros and become the padding.
// DWORDS: rows of whole dwords, loaded through a descriptor that ends with the
// row.  Else (bf16 rows that start or end at odd elements) the chunks past the
// last whole one are loaded to end with the row and shifted into place.  Bound
// by the bytes of a large x (131072 x 2048 fp32: 224 us, 6.0 TB/s), by latency
// for a few rows.
template <typename T, int WPR, int NV, bool DWORDS>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T* x, int64_t ldx, int64_t M, int K,
                                                            int Kp, int8_t* q, float* scale) {
  using C = Chunk<T>;
  __shared__ uint32_t s_top[4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t row = int64_t(blockIdx.x) * (4 / WPR) + wave / WPR;
  if (row >= M) return;  // (WPR == 4: never)
  const int c0 = wave % WPR * 64 + lane;
  const T* src = x + row * ldx;
  u32x4 w[NV];
  if constexpr (DWORDS) {
    const auto rsrc =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(src), 0, K * int(sizeof(T)), 0x00020000);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      w[j] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, (c0 + j * 64 * WPR) * 16, 0, 2);
  } else {
    const int last = K - C::kSize;  // >= 0
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (c0 + j * 64 * WPR) * C::kSize;
      w[j] = load16(src + (k < last ? k : last));
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int past = (c0 + j * 64 * WPR) * C::kSize - last;
      if (past > 0) w[j] = past < C::kSize ? from_element<T>(w[j], past) : u32x4{};
    }
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
    if (k < Kp) store_codes(codes, dst + k);
  }
}

// Rows of up to NV x LPR x 16 bytes, padding included: LPR lanes each, two or
// four rows to a wave.  Measured (us, this kernel / a wave per row): bf16
// 131072 x 21 11.0 / 52, 131072 x 256 19.6 / 53, 131072 x 512 30.7 / 54, 256 x 256
// 3.4 / 3.3; fp32 131072 x 128 16.4 / 33, 131072 x 256 25.2 / 35.
template <typename T, int LPR, int NV>
__global__ __launch_bounds__(256) void quantize_short_rows_kernel(const T* x, int64_t ldx, int64_t M, int K,
                                                                  int Kp, int8_t* q, float* scale) {
  using C = Chunk<T>;
  constexpr int V = C::kSize;
  const int64_t row = (int64_t(blockIdx.x) * 256 + threadIdx.x) / LPR;
  const int c = threadIdx.x % LPR;
  const T* src = x + (row < M ? row : M - 1) * ldx;
  u32x4 w[NV] = {};
  if (K >= V) {
    const int last = K - V;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (c + j * LPR) * V;
      w[j] = load16(src + (k < last ? k : last));
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int past = (c + j * LPR) * V - last;
      if (past > 0) w[j] = past < V ? from_element<T>(w[j], past) : u32x4{};
    }
  } else if (c == 0) {
#pragma unroll
    for (int e = 0; e < V - 1; ++e) {
      const uint32_t x = __float_as_uint(load_f32(src + (e < K ? e : 0)));  // bf16: its bits on top
      if constexpr (sizeof(T) == 4)
        w[0][e] = e < K ? x : 0;
      else
        w[0][e / 2] |= (e < K ? x : 0) >> (e % 2 ? 0 : 16);
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t t = C::top(w[j]);
    top = top > t ? top : t;
  }
#pragma unroll
  for (int d = 1; d < LPR; d <<= 1) {
    const uint32_t o = __shfl_xor(top, d);
    top = top > o ? top : o;
  }
  const float s = row_scale(top), d = s == 0.0f ? 1.0f : s;
  const bool plain = __builtin_amdgcn_ballot_w64(!divides_plainly(d)) == 0;  // all of the wave's rows
  const float r = plain ? __fdiv_rn(1.0f, d) : 0.0f;
  if (row >= M) return;
  if (c == 0) scale[row] = s;
  const int width = NV == 1 ? LPR * V : Kp;
  auto emit = [&](float by, bool fast) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (c + j * LPR) * V;
      uint32_t codes[V / 4];
      C::codes(w[j], by, r, fast, codes);
      if (k < width) store_codes(codes, q + row * width + k);
    }
  };
  if (plain)  // the stores within, or the compiler computes both sides
    emit(d, true);
  else
    emit(s, false);
}

// Rows too long for registers: one per workgroup, read twice (the second time
// from the caches).  Also of rows without elements.
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
// threads owns TPR x 16 bytes of columns, TPR threads to a row; a thread holds
// four consecutive rows of a pass over 4096 / TPR, so that it writes four codes of
// a column as one dword.  Up to NP passes all of W is read once; beyond, its
// first part twice (MORE).  Neighbouring workgroups share lines, so each XCD
// takes a contiguous range.  All of a CU's loads are in flight at once, its
// products and stores after them: 2048 x 4096 fp32 11.5 us, 3.6 TB/s, of which
// the bytes take 6.9 and the launch 2.
template <typename T, int TPR, int NP, bool MORE>
__global__ __launch_bounds__(1024) void quantize_columns_kernel(const T* W, int64_t ldw, int64_t K, int64_t N,
                                                                int64_t Kp, int8_t* q, float* scale) {
  using C = Chunk<T>;
  constexpr int V = C::kSize, kCols = TPR * V, kPass = 4096 / TPR;
  __shared__ uint32_t s_top[16][kCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t per = gridDim.x / 8;
  const uint32_t tile = blockIdx.x < per * 8 ? (blockIdx.x % 8) * per + blockIdx.x / 8 : blockIdx.x;
  const int64_t n0 = int64_t(tile) * kCols;
  const int c = (threadIdx.x % TPR) * V, g = threadIdx.x / TPR;
  // A chunk that would pass the last column is loaded to end with it (N >= V)
  // and shifted into place.
  const int64_t n = n0 + c < N - V ? n0 + c : N - V;
  const int past = int(n0 + c - n);
  u32x4 w[NP][4];
  auto load = [&](int64_t base) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t k = base + p * kPass + 4 * g + i;
        w[p][i] = u32x4{};
        if (k < K) w[p][i] = load16(W + k * ldw + n);
      }
    if (past > 0 && past < V) {
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[p][i] = from_element<T>(w[p][i], past);
    }
  };
  int64_t base = 0;
  uint32_t top[V] = {};
  for (;; base += NP * kPass) {
    load(base);
#pragma unroll
    for (int e = 0; e < V; ++e)
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t b = abs_bits(C::get(w[p][i], e));
          top[e] = top[e] > b ? top[e] : b;
        }
    if (!MORE || base + NP * kPass >= K) break;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int d = TPR; d < 64; d <<= 1) {
      const uint32_t o = __shfl_xor(top[e], d);
      top[e] = top[e] > o ? top[e] : o;
    }
  }
  if (lane < TPR) {
#pragma unroll
    for (int e = 0; e < V; ++e) s_top[wave][c + e] = top[e];
  }
  __syncthreads();
  bool rare = false;
  if (threadIdx.x < kCols) {
    uint32_t t = 0;
#pragma unroll
    for (int v = 0; v < 16; ++v) t = t > s_top[v][threadIdx.x] ? t : s_top[v][threadIdx.x];
    s_top[0][threadIdx.x] = t;  // (only this thread reads the column)
    const float s = row_scale(t);
    if (n0 + threadIdx.x < N) {
      scale[n0 + threadIdx.x] = s;
      rare = s != 0.0f && !divides_plainly(s);
    }
  }
  // A column whose scale is not finite or at an end of the fp32 range: all of
  // them once more from memory, in little code (unrolled beside the other it
  // doubled the kernel).
  if (__syncthreads_or(rare)) {
    for (int e = threadIdx.x / 64; e < kCols && n0 + e < N; e += 16) {
      const float s = row_scale(s_top[0][e]);
      uint32_t* dst = reinterpret_cast<uint32_t*>(q + (n0 + e) * Kp);
      for (int64_t k = int64_t(lane) * 4; k < Kp; k += 256) {
        uint32_t v = 0;
        for (int i = 0; i < 4; ++i)
          if (k + i < K) v |= code(load_f32(W + (k + i) * ldw + n0 + e), s, s > 0.0f) << (8 * i);
        dst[k / 4] = v;
      }
    }
    return;
  }
  for (;; base -= NP * kPass) {  // the last part first: it is in registers
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (n0 + c + e >= N) break;
      float s = row_scale(s_top[0][c + e]);
      s = s == 0.0f ? 1.0f : s;  // a column of zeros
      const float r = __fdiv_rn(1.0f, s);
      int8_t* dst = q + (n0 + c + e) * Kp;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int64_t k = base + p * kPass + 4 * g;
        if (k >= Kp) break;
        uint32_t v = 0;
#pragma unroll
        for (int i = 3; i >= 0; --i)
          v = (v << 8) | (uint32_t(int(rintf(divided(C::get(w[p][i], e), s, r)))) & 0xFFu);
        *reinterpret_cast<uint32_t*>(dst + k) = v;
      }
    }
    if (!MORE || base == 0) break;
    load(base - NP * kPass);
  }
}

// Columns of a W that is narrower than 16 bytes, or has no rows: a workgroup
// owns kColTile columns, finds their largest magnitudes over all K rows, then
// reads the rows again.
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

template <typename T, int WPR, bool DWORDS>
void launch_rows(int nv, int64_t M, int K, int Kp, const T* x, int64_t ldx, int8_t* q, float* scale,
                 hipStream_t stream) {
  const dim3 grid{uint32_t((M * WPR + 3) / 4)}, block{256};
  auto run = [&](auto* kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, x, ldx, M, K, Kp, q, scale); };
  if (nv <= 2) run(quantize_rows_kernel<T, WPR, 2, DWORDS>);
  else if (nv <= 4) run(quantize_rows_kernel<T, WPR, 4, DWORDS>);
  else if (nv <= 8) run(quantize_rows_kernel<T, WPR, 8, DWORDS>);
  else run(quantize_rows_kernel<T, WPR, 16, DWORDS>);
}

// Chunks per lane that the kernels for whole rows go up to.
constexpr int kMaxChunks = 16;
// Rows of more than four chunks per lane (4 KB), up to so many, are split over four
// waves.  Measured (us, four waves / one per row): 1024 x 2048 fp32 3.1 / 3.4,
// 2048 x 2048 fp32 4.2 / 4.6, 4096 x 2048 fp32 8.2 / 8.1, 1024 x 4096 bf16 3.6 / 4.1;
// 256 x 2048 bf16 2.5 / 2.6, 1024 x 2048 bf16 3.8 / 2.8, 1024 x 512 bf16 3.1 / 2.3.
constexpr int64_t kFewRows = 2048;

template <typename T, bool DWORDS>
void launch_rows(int64_t M, int64_t K, int64_t Kp, int64_t chunks, const T* x, int64_t ldx, int8_t* q, float* scale,
                 hipStream_t stream) {
  if ((M <= kFewRows && chunks > 64 * 4) || chunks > 64 * kMaxChunks)
    launch_rows<T, 4, DWORDS>(int((chunks + 255) / 256), M, int(K), int(Kp), x, ldx, q, scale, stream);
  else
    launch_rows<T, 1, DWORDS>(int((chunks + 63) / 64), M, int(K), int(Kp), x, ldx, q, scale, stream);
}

template <typename T>
void launch_rows(int64_t M, int64_t K, const T* x, int64_t ldx, int8_t* q, float* scale,
                 hipStream_t stream) {
  const int64_t Kp = quantized_row_bytes(K);
  const int64_t chunks = (Kp * int64_t(sizeof(T)) + 15) / 16;  // Kp: the padding is written too
  const bool dwords = sizeof(T) == 4 || ((ldx % 2 == 0 || M == 1) && K % 2 == 0 && aligned(x, 4));
  if (K > 0 && chunks <= 64) {
    auto run = [&](auto* kernel, int64_t lanes) {
      hipLaunchKernelGGL(kernel, dim3(uint32_t((M * lanes + 255) / 256)), dim3(256), 0, stream, x, ldx, M, int(K),
                         int(Kp), q, scale);
    };
    if (chunks == 32) {  // the chunks of 128 codes, once or twice
      run(quantize_short_rows_kernel<T, 32, 1>, 32);
    } else if (chunks > 32) {
      run(quantize_short_rows_kernel<T, 32, 2>, 32);
    } else if constexpr (sizeof(T) == 2) {
      run(quantize_short_rows_kernel<T, 16, 1>, 16);
    }
    return;
  }
  if (K == 0 || chunks > 4 * 64 * kMaxChunks) {
    hipLaunchKernelGGL(quantize_any_rows_kernel<T>, dim3(uint32_t(M)), dim3(256), 0, stream, x, ldx, K, Kp, q,
                       scale);
    return;
  }
  if constexpr (sizeof(T) == 2) {
    if (!dwords) return launch_rows<T, false>(M, K, Kp, chunks, x, ldx, q, scale, stream);
  }
  launch_rows<T, true>(M, K, Kp, chunks, x, ldx, q, scale, stream);
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
  if (K == 0 || N < Chunk<T>::kSize) {
    hipLaunchKernelGGL(quantize_any_columns_kernel<T>, dim3(uint32_t((N + kColTile - 1) / kColTile)), dim3(256), 0,
                       stream, W, ldw, K, N, Kp, q, scale);
    return;
  }
  auto run = [&](auto* kernel, int tpr) {
    const int64_t cols = tpr * Chunk<T>::kSize;
    hipLaunchKernelGGL(kernel, dim3(uint32_t((N + cols - 1) / cols)), dim3(1024), 0, stream, W, ldw, K, N, Kp, q,
                       scale);
  };
  // 64 bytes of columns per workgroup where that gives every CU one or the rows
  // are few, else 32 (also where 64 bytes of bf16 would not fit the registers).
  // Measured (us, 64 / 32 bytes): 2048 x 4096 fp32 12.7 / 14.3, 4096 x 4096 fp32
  // 24.0 / 34.4, 2048 x 1000 fp32 9.3 / 8.1; 2048 x 8192 bf16 17.1 / 18.1, 2048 x
  // 4096 bf16 13.7 / 12.2, 200 x 8000 bf16 7.2 / 9.6.
  if (K <= 512 || (N >= 256 * 4 * Chunk<T>::kSize && (sizeof(T) == 4 || K <= 2048))) {
    if (K <= 1024) {
      run(quantize_columns_kernel<T, 4, 1, false>, 4);
    } else if (K <= 2048) {
      run(quantize_columns_kernel<T, 4, 2, false>, 4);
    } else if constexpr (sizeof(T) == 4) {
      if (K <= 4096)
        run(quantize_columns_kernel<T, 4, 4, false>, 4);
      else
        run(quantize_columns_kernel<T, 4, 4, true>, 4);
    }
  } else {
    if (K <= 2048)
      run(quantize_columns_kernel<T, 2, 1, false>, 2);
    else if (K <= 4096)
      run(quantize_columns_kernel<T, 2, 2, false>, 2);
    else
      run(quantize_columns_kernel<T, 2, 2, true>, 2);
  }
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
