// Scales and codes of the symmetric 8-bit quantisation (quant.hip says what
// they are), shared by the kernels that write codes to memory and those that
// quantise their own operand.
#pragma once

#include "device_util.hpp"

namespace sr {

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

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// The elements of 16 bytes of fp32 or bf16 (uint16_t).
template <typename T>
struct Chunk {
  static constexpr int kSize = 16 / sizeof(T);
  static __device__ __forceinline__ uint32_t top(u32x4 w) {  // of their magnitudes
    uint32_t t = 0;
#pragma unroll
    for (int e = 0; e < kSize; ++e) {
      const uint32_t b = abs_bits(get(w, e));
      t = t > b ? t : b;
    }
    return t;
  }
  // Their codes, four to a dword; r = 1 / s where divides_plainly(s).
  static __device__ __forceinline__ void codes(u32x4 w, float s, float r, bool plain, uint32_t (&c)[kSize / 4]) {
    if (plain) {
#pragma unroll
      for (int d = 0; d < kSize / 4; ++d) {
        c[d] = 0;
        // |x| <= 127 s (1 + 2^-24), so the quotient rounds to 127 at most.
#pragma unroll
        for (int e = 3; e >= 0; --e)
          c[d] = (c[d] << 8) | (uint32_t(int(rintf(divided(get(w, d * 4 + e), s, r)))) & 0xFFu);
      }
    } else {
#pragma unroll
      for (int d = 0; d < kSize / 4; ++d) {
        c[d] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) c[d] |= code(get(w, d * 4 + e), s, s > 0.0f) << (8 * e);
      }
    }
  }
  static __device__ __forceinline__ float get(u32x4 w, int e) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    return __uint_as_float(e % 2 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
  }
};

}  // namespace sr
