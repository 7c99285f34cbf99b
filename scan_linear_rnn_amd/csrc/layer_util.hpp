// Device pieces shared by the kernels of the selective scan (selective.hip,
// selective_bwd.hip), the short convolution (conv.hip) and the norm (norm.hip).
#pragma once

#include <cfloat>

#include "device_util.hpp"
#include "internal.hpp"

namespace sr {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(uint16_t x) { return __uint_as_float(uint32_t(x) << 16); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float x) { return uint16_t(bf16_pair(x, 0.0f)); }

// The element at a byte offset from an address that all lanes share: loads take the
// two as they are.
template <typename T>
__device__ __forceinline__ T* at_byte(T* base, uint32_t offset) {
  using Byte = std::conditional_t<std::is_const_v<T>, const char, char>;
  return reinterpret_cast<T*>(reinterpret_cast<Byte*>(base) + offset);
}

// N neighbouring elements at any element: global loads and stores take any
// address that is a multiple of the element's size.
template <int N, typename T>
__device__ __forceinline__ void load_n(const T* p, float (&v)[N]) {
  if constexpr (sizeof(T) == 4) {
    __builtin_memcpy(v, __builtin_assume_aligned(p, 4), N * 4);
  } else {
    if constexpr (N == 1) {
      v[0] = to_f32(*p);
      return;
    }
    uint32_t w[(N + 1) / 2];
    __builtin_memcpy(w, __builtin_assume_aligned(p, 2), N * 2);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <int N, typename T>
__device__ __forceinline__ void store_n(T* p, const float (&v)[N]) {
  if constexpr (sizeof(T) == 4) {
    __builtin_memcpy(__builtin_assume_aligned(p, 4), v, N * 4);
  } else {
    if constexpr (N == 1) {
      *p = from_f32<T>(v[0]);
      return;
    }
    uint32_t w[(N + 1) / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    __builtin_memcpy(__builtin_assume_aligned(p, 2), w, N * 2);
  }
}

// The first n of N elements; zeros for the others.
template <int N, typename T>
__device__ __forceinline__ void load_some(const T* p, int n, float (&v)[N]) {
  if (n >= N) {
    load_n(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
  }
}
template <int N, typename T>
__device__ __forceinline__ void store_some(T* p, int n, const float (&v)[N]) {
  if (n >= N) {
    store_n(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

// Q neighbouring elements as they stand in memory, for loads that are on the way
// while something else is computed: their conversion waits for them.
template <typename T, int Q>
struct Raw {
  static constexpr int kWords = (Q * int(sizeof(T)) + 3) / 4;
  uint32_t w[kWords];
};
// kWhole: all Q exist; else the last of the n >= 1 is repeated (and waited for).
template <bool kWhole, typename T, int Q>
__device__ __forceinline__ void load_raw(const T* p, int n, Raw<T, Q>& r) {
  if constexpr (Q * sizeof(T) == 2) {
    r.w[0] = *p;
  } else if constexpr (kWhole) {
    __builtin_memcpy(r.w, __builtin_assume_aligned(p, sizeof(T)), sizeof(r.w));
  } else {
    T v[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) v[i] = p[i < n ? i : n - 1];
    __builtin_memcpy(r.w, v, sizeof(r.w));
  }
}
template <int Q>
__device__ __forceinline__ void values(const Raw<float, Q>& r, float (&v)[Q]) {
#pragma unroll
  for (int i = 0; i < Q; ++i) v[i] = __uint_as_float(r.w[i]);
}
template <int Q>
__device__ __forceinline__ void values(const Raw<uint16_t, Q>& r, float (&v)[Q]) {
#pragma unroll
  for (int i = 0; i < Q; ++i) v[i] = __uint_as_float(i % 2 ? r.w[i / 2] & 0xFFFF0000u : r.w[i / 2] << 16);
}

// Stores of n elements at a byte offset from an address that all lanes share,
// dropped where the offset is kNowhere: without a branch, so that the loads in
// flight can be told from the stores behind them and waited for alone.  The
// elements are aligned as a whole.
constexpr uint32_t kNowhere = 0x80000000u;  // past the 2^31 - 1 bytes that a store reaches, with what it writes
template <typename T, int N>
__device__ __forceinline__ void store_at(T* base, uint32_t offset, const float (&v)[N]) {
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(base, 0, 0x7FFFFFFF, 0x00020000);
  if constexpr (sizeof(T) == 2) {
    if constexpr (N == 1) {
      __builtin_amdgcn_raw_buffer_store_b16(from_f32<uint16_t>(v[0]), rsrc, int(offset), 0, 0);
    } else if constexpr (N == 2) {
      __builtin_amdgcn_raw_buffer_store_b32(bf16_pair(v[0], v[1]), rsrc, int(offset), 0, 0);
    } else {
      typedef unsigned int Two __attribute__((ext_vector_type(2)));
      __builtin_amdgcn_raw_buffer_store_b64(Two{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}, rsrc, int(offset), 0, 0);
    }
  } else {
    typedef unsigned int Two __attribute__((ext_vector_type(2)));
    typedef unsigned int Four __attribute__((ext_vector_type(4)));
    const auto bits = [&](int i) { return __float_as_uint(v[i]); };
    if constexpr (N == 1)
      __builtin_amdgcn_raw_buffer_store_b32(bits(0), rsrc, int(offset), 0, 0);
    else if constexpr (N == 2)
      __builtin_amdgcn_raw_buffer_store_b64(Two{bits(0), bits(1)}, rsrc, int(offset), 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b128(Four{bits(0), bits(1), bits(2), bits(3)}, rsrc, int(offset), 0, 0);
  }
}

// A rate of the selective scan, and the factor of a step in its power of two: never minus
// infinity, so that the steps of zero behind a sequence's end leave the state for any rate.
__device__ __forceinline__ float bounded(float a) { return a < -FLT_MAX ? -FLT_MAX : a; }
__device__ __forceinline__ float rate2(float a) { return bounded(a * kLog2e); }

// 4^x h + e, the decay of many tokens: its factor may leave the fp32 range where the
// product does not (a small state that grows), so it comes in two halves of x each.
__device__ __forceinline__ float decayed(float x, float h, float e) {
  const float half = __builtin_amdgcn_exp2f(x);
  return fmaf(half, half * h, e);
}
__device__ __forceinline__ float half_rate2(float a) { return bounded(a * (0.5f * kLog2e)); }

// log(1 + e^x) = max(x, 0) + log1p(e), e = e^-|x|.  With u the rounded 1 + e, log1p(e) = log(u) +
// (e - (u - 1)) / u; u's rounding error e - (u - 1) is exact, and what its division by u
// changes is far below the sum's last place.  The exponent |x| log2 e is rounded (the constant
// too), so the result is off by up to (2 |x| + 8) 2^-24 of it.
__device__ __forceinline__ float softplus_f(float x) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(x) * kLog2e);
  const float u = 1.0f + e;
  return fmaxf(x, 0.0f) + fmaf(__builtin_amdgcn_logf(u), kLn2, e - (u - 1.0f));  // (a NaN is in e)
}

// 1 / (1 + e^-x), off by up to (2 |x| + 6) 2^-24 of it by the rounded exponent.
__device__ __forceinline__ float logistic_f(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * kLog2e));
}

// Lane n of each row of 16 lanes, in all lanes of the row: multiplications take
// it as an operand of their own.
template <int n>
__device__ __forceinline__ float of_row(float x) {
  return __uint_as_float(
      uint32_t(__builtin_amdgcn_mov_dpp(int(__float_as_uint(x)), 0x150 + n, 0xF, 0xF, true)));
}
// of_row<n>(m) x.  (Opaque behind it, so that products of several numbers are not made
// vectors of: those would take the operand from a register of its own.)
template <int n>
__device__ __forceinline__ float row_times(float m, float x) {
  float y = of_row<n>(m) * x;
  asm("" : "+v"(y));
  return y;
}
// sum_i m[i][n] x[i] with m[i][n] in lane n of each row of 16.  (The compiler does not
// put such an operand into fused multiply-adds by itself.  The two wait states are
// those between a vector instruction's result and its use across lanes.)
template <int n>
__device__ __forceinline__ float row_dot(const float (&m)[1], const float (&x)[1]) {
  return row_times<n>(m[0], x[0]);
}
template <int n>
__device__ __forceinline__ float row_dot(const float (&m)[2], const float (&x)[2]) {
  float sum;
  asm("s_nop 1\n\t"
      "v_mul_f32_dpp %0, %1, %3 row_newbcast:%5 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %0, %2, %4 row_newbcast:%5 row_mask:0xf bank_mask:0xf"
      : "=&v"(sum)
      : "v"(m[0]), "v"(m[1]), "v"(x[0]), "v"(x[1]), "i"(n));
  return sum;
}
// Two of them, n and n + 1: neither has to wait for its own last product.
template <int n>
__device__ __forceinline__ void row_dots(const float (&m)[1], const float (&x)[1], const float (&y)[1], float& sx, float& sy) {
  sx = row_times<n>(m[0], x[0]);
  sy = row_times<n + 1>(m[0], y[0]);
}
template <int n>
__device__ __forceinline__ void row_dots(const float (&m)[2], const float (&x)[2], const float (&y)[2], float& sx, float& sy) {
  asm("s_nop 1\n\t"
      "v_mul_f32_dpp %0, %2, %4 row_newbcast:%8 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %1, %2, %6 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %0, %3, %5 row_newbcast:%8 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %1, %3, %7 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
      : "=&v"(sx), "=&v"(sy)
      : "v"(m[0]), "v"(m[1]), "v"(x[0]), "v"(x[1]), "v"(y[0]), "v"(y[1]), "i"(n), "i"(n + 1));
}
template <int n>
__device__ __forceinline__ void row_dots(const float (&m)[4], const float (&x)[4], const float (&y)[4], float& sx, float& sy) {
  asm("s_nop 1\n\t"
      "v_mul_f32_dpp %0, %2, %6 row_newbcast:%14 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %1, %2, %10 row_newbcast:%15 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %0, %3, %7 row_newbcast:%14 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %1, %3, %11 row_newbcast:%15 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %0, %4, %8 row_newbcast:%14 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %1, %4, %12 row_newbcast:%15 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %0, %5, %9 row_newbcast:%14 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %1, %5, %13 row_newbcast:%15 row_mask:0xf bank_mask:0xf"
      : "=&v"(sx), "=&v"(sy)
      : "v"(m[0]), "v"(m[1]), "v"(m[2]), "v"(m[3]), "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]), "v"(y[0]), "v"(y[1]),
        "v"(y[2]), "v"(y[3]), "i"(n), "i"(n + 1));
}

template <int n>
__device__ __forceinline__ void row_dots(const float (&m)[8], const float (&x)[8], const float (&y)[8], float& sx, float& sy) {
  const auto half = [](const float (&v)[8], int at, float (&to)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = v[at + i];
  };
  float a[4], b[4], c[4], bx, by;
  half(m, 0, a), half(x, 0, b), half(y, 0, c);
  row_dots<n>(a, b, c, sx, sy);
  half(m, 4, a), half(x, 4, b), half(y, 4, c);
  row_dots<n>(a, b, c, bx, by);
  sx += bx;
  sy += by;
}

// y[i] += m[i][n] x with m[i][n] in lane n of each row of 16.
template <int n>
__device__ __forceinline__ void row_add(const float (&m)[1], float x, float (&y)[1]) {
  y[0] += row_times<n>(m[0], x);
}
template <int n>
__device__ __forceinline__ void row_add(const float (&m)[2], float x, float (&y)[2]) {
  asm("s_nop 1\n\t"
      "v_fmac_f32_dpp %0, %2, %4 row_newbcast:%5 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %1, %3, %4 row_newbcast:%5 row_mask:0xf bank_mask:0xf"
      : "+&v"(y[0]), "+&v"(y[1])
      : "v"(m[0]), "v"(m[1]), "v"(x), "i"(n));
}
template <int n>
__device__ __forceinline__ void row_add(const float (&m)[4], float x, float (&y)[4]) {
  asm("s_nop 1\n\t"
      "v_fmac_f32_dpp %0, %4, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %1, %5, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %2, %6, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %3, %7, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
      : "+&v"(y[0]), "+&v"(y[1]), "+&v"(y[2]), "+&v"(y[3])
      : "v"(m[0]), "v"(m[1]), "v"(m[2]), "v"(m[3]), "v"(x), "i"(n));
}

template <int n>
__device__ __forceinline__ void row_add(const float (&m)[8], float x, float (&y)[8]) {
  asm("s_nop 1\n\t"
      "v_fmac_f32_dpp %0, %8, %16 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %1, %9, %16 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %2, %10, %16 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %3, %11, %16 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %4, %12, %16 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %5, %13, %16 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %6, %14, %16 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %7, %15, %16 row_newbcast:%17 row_mask:0xf bank_mask:0xf"
      : "+&v"(y[0]), "+&v"(y[1]), "+&v"(y[2]), "+&v"(y[3]), "+&v"(y[4]), "+&v"(y[5]), "+&v"(y[6]), "+&v"(y[7])
      : "v"(m[0]), "v"(m[1]), "v"(m[2]), "v"(m[3]), "v"(m[4]), "v"(m[5]), "v"(m[6]), "v"(m[7]), "v"(x), "i"(n));
}

// Calls f with 0 .. n - 1 as constants.
template <int n, typename F, int i = 0>
__device__ __forceinline__ void unrolled(F f) {
  if constexpr (i < n) {
    f(std::integral_constant<int, i>{});
    unrolled<n, F, i + 1>(f);
  }
}

// Sums of the columns of parts [rows][cols] in fp32, always in the same order: 16
// threads per column, each its rows in turn, eight loads ahead.  out(column, sum).
template <typename Out>
__device__ __forceinline__ void column_sums(const float* parts, int64_t rows, int64_t cols, Out out) {
  __shared__ float s_sum[16][64];
  const int lane = threadIdx.x & 63, part = threadIdx.x >> 6;
  const int64_t c = int64_t(blockIdx.x) * 64 + lane;
  float sum = 0.0f;
  if (c < cols) {
    int64_t r = part;
    for (; r + 7 * 16 < rows; r += 8 * 16) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = parts[(r + j * 16) * cols + c];
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += v[j];
    }
    for (; r < rows; r += 16) sum += parts[r * cols + c];
  }
  s_sum[part][lane] = sum;
  __syncthreads();
  if (part == 0 && c < cols) {
#pragma unroll
    for (int j = 1; j < 16; ++j) sum += s_sum[j][lane];
    out(c, sum);
  }
}

// The offset in bytes of element i of a tile's row t.  (Rows that may be further apart than 32 bits hold
// are rows of one token, t = 0.)
template <typename T>
__device__ __forceinline__ uint32_t row_bytes(int t, int64_t ld, int i) {
  return (uint32_t(t) * uint32_t(ld) + uint32_t(i)) * uint32_t(sizeof(T));
}

constexpr int kTile = kSelectiveTile;  // tokens per tile
constexpr int kLanes = 64;             // channels per workgroup

// Which 64 channels of which sequence and chunk a workgroup has.
struct Place {
  int64_t b;
  int group, chunk;
  int64_t c0;  // first channel
  int width;   // channels, 1 to 64
  int tile;    // of the group
};
__device__ __forceinline__ Place place_of(const SelectiveRequest& P) {
  Place p;
  const uint32_t tiles = uint32_t(P.tiles_per_group) * uint32_t(P.G);
  uint32_t i = blockIdx.x;
  const uint32_t t = i % tiles;
  i /= tiles;
  p.b = i % uint32_t(P.B);
  p.chunk = int(i / uint32_t(P.B));
  p.group = int(t) / P.tiles_per_group;
  p.tile = int(t) % P.tiles_per_group;
  const int64_t per = P.D / P.G;
  p.c0 = p.group * per + int64_t(p.tile) * kLanes;
  const int64_t left = per - int64_t(p.tile) * kLanes;
  p.width = int(left < kLanes ? left : kLanes);
  return p;
}

// Tokens of sequence b.
__device__ __forceinline__ int64_t length_of(const SelectiveRequest& P, int64_t b) {
  if (P.lengths == nullptr) return P.T;
  const int64_t n = P.lengths[b];
  return n < 0 ? 0 : n < P.T ? n : P.T;
}

}  // namespace sr
