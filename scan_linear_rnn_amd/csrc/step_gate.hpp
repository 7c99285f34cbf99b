// The minGRU update of one (row, channel) in a single-token step.  The gates
// and the interpolation are shared by the step kernels' epilogues (gemm.hip,
// gemm_i8.hip); carried_state is the fp32 step's, the step on codes scales four
// channels at a time (decayed in gemm_i8.hip).
#pragma once

#include "internal.hpp"

namespace sr {

// sigma(k) from e = e^{-|k|}: 1/(1+e) for k >= 0, e/(1+e) below.
__device__ __forceinline__ float sigmoid_f(float k) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float e = __builtin_amdgcn_exp2f(-fabsf(k) * kLog2e);
  const float big = __builtin_amdgcn_rcpf(1.0f + e);
  return k >= 0.0f ? big : e * big;
}

__device__ __forceinline__ float g_act(float p) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float ep = __builtin_amdgcn_exp2f(fminf(p, 0.0f) * kLog2e);
  return p >= 0.0f ? p + 0.5f : ep * __builtin_amdgcn_rcpf(1.0f + ep);
}

// The carried state entering the step for one (row, channel): h_prev (zero
// when absent), with time decay first scaled by exp(-min(rate_d * gap_row,
// 1e4)) (the token boundary comes before the token's write; exp(-1e4) is
// zero in float32, so the clamp changes no value and only marks saturation).
// Params has h_prev, D_h and the decay's rate, gap, log1p_gap and saturated.
template <class Params>
__device__ __forceinline__ float carried_state(const Params& P, int64_t row, int64_t d) {
  float hp = P.h_prev ? P.h_prev[row * P.D_h + d] : 0.0f;
  if (P.rate != nullptr) {
    constexpr float kClamp = 1.0e4f, kLog2e = 1.4426950408889634f;
    const float gap = P.log1p_gap ? log1pf(P.gap[row]) : P.gap[row];
    const float e = P.rate[d] * gap;
    if (e > kClamp && P.saturated != nullptr)
      __hip_atomic_fetch_or(P.saturated, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    hp *= __builtin_amdgcn_exp2f(fminf(e, kClamp) * -kLog2e);
  }
  return hp;
}

// h_next = (1 - z) h + z g(p) with z = sigma(k), h the carried state,
// evaluated as the interpolation h + z (g(p) - h): the complement 1 - z is
// never rounded on its own, so a gate that keeps almost all of the state
// (z tiny) moves it by exactly z times the gap to the candidate, and h = g(p)
// is a fixed point.
__device__ __forceinline__ float step_value(float k, float p, float h) {
  return fmaf(sigmoid_f(k), g_act(p) - h, h);
}

}  // namespace sr
