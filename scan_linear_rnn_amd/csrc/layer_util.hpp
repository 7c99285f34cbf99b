// Device pieces shared by the kernels of the selective scan (selective.hip,
// selective_bwd.hip), the short convolution (conv.hip) and the norm (norm.hip).
#pragma once

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
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float x) { return uint16_t(bf16_bits(x)); }

// N neighbouring elements at any element: global loads and stores take any
// address that is a multiple of the element's size.
typedef float f32x4 __attribute__((ext_vector_type(4)));
template <int N, typename T>
__device__ __forceinline__ void load_n(const T* p, float (&v)[N]) {
  if constexpr (sizeof(T) == 4) {
    __builtin_memcpy(v, __builtin_assume_aligned(p, 4), N * 4);
  } else {
    uint32_t w[N / 2];
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
    uint32_t w[N / 2];
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
template <typename T>
__device__ __forceinline__ f32x4 load4(const T* p, int n) {
  float v[4];
  load_some(p, n, v);
  return f32x4{v[0], v[1], v[2], v[3]};
}
template <typename T>
__device__ __forceinline__ void store4(T* p, f32x4 v, int n) {
  const float w[4] = {v[0], v[1], v[2], v[3]};
  store_some(p, n, w);
}

// A weight of either type.
__device__ __forceinline__ float weight_at(const void* w, sr_dtype dtype, int64_t i) {
  return dtype == SR_BF16 ? to_f32(static_cast<const uint16_t*>(w)[i]) : static_cast<const float*>(w)[i];
}

// log(1 + e^x) to a few ulps for any x: max(x, 0) + log1p(e^-|x|), the
// logarithm by W. Kahan's correction log1p(e) = log(u) e / (u - 1) with u the
// rounded 1 + e, which undoes u's rounding error.
__device__ __forceinline__ float softplus_f(float x) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(x) * kLog2e);
  const float u = 1.0f + e, d = u - 1.0f;
  const float l = d > 0.0f ? __builtin_amdgcn_logf(u) * (kLn2 * e) * __builtin_amdgcn_rcpf(d) : e;
  return x != x ? x : fmaxf(x, 0.0f) + l;
}

// 1 / (1 + e^-x), to a few ulps.
__device__ __forceinline__ float logistic_f(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * kLog2e));
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

constexpr int kTile = kSelectiveTile;  // tokens per tile
constexpr int kLanes = 64;             // channels per workgroup
constexpr int kNS = 4;                 // states per lane

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
