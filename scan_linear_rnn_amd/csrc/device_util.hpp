// Small device helpers shared by the 8-bit and AdamW kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace sr {

constexpr uint32_t kF32InfBits = 0x7F800000u;

// fp32 to bf16, to nearest with ties to even; NaNs stay NaN.
__device__ __forceinline__ uint32_t bf16_bits(float x) {
  const uint32_t u = __float_as_uint(x);
  if ((u & 0x7FFFFFFFu) > kF32InfBits) return 0x7FC0u;
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// Two fp32 as packed bf16, rounded as above.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// Bits of |x|: ordered like the values, infinities and then NaNs on top.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The largest value of a wave (uniform): lane 15 of each row of 16 collects
// the row, rows 1 and 3 their predecessor, lane 63 the first half.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto take = [&](auto ctrl) {
    const uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), decltype(ctrl)::value, 0xF, 0xF, false));
    v = v > o ? v : o;
  };
  take(std::integral_constant<int, 0x111>{});  // row_shr 1, 2, 4, 8
  take(std::integral_constant<int, 0x112>{});
  take(std::integral_constant<int, 0x114>{});
  take(std::integral_constant<int, 0x118>{});
  take(std::integral_constant<int, 0x142>{});  // row_bcast 15, 31
  take(std::integral_constant<int, 0x143>{});
  return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}

// x / s for a scale s away from the ends of the fp32 range, r = 1 / s
// correctly rounded: the first correction brings the product within an ulp,
// the second makes it the IEEE quotient (P. Markstein, Computation of
// elementary functions on the IBM RISC System/6000, 1990), in five
// instructions instead of the division's ten.
__device__ __forceinline__ float divided(float x, float s, float r) {
  float q = x * r;
  q = fmaf(fmaf(-q, s, x), r, q);
  return fmaf(fmaf(-q, s, x), r, q);
}
__device__ __forceinline__ bool divides_plainly(float s) { return s > 0x1p-96f && s < 0x1p96f; }

}  // namespace sr
