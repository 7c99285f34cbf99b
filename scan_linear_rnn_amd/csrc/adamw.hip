// One AdamW step over many tensors in few launches, states in fp32 or in 8
// bits.  For each element, with the step's number t and c1 = 1 - b1^t,
// c2 = 1 - b2^t:
//
//     g = grad * grad_scale
//     m = b1 m + (1 - b1) g        v = b2 v + (1 - b2) g^2
//     p = p (1 - lr wd) - (lr / c1) m / (sqrt(v) / sqrt(c2) + eps)
//
// in fp32 whatever the tensors' types; p is rounded once when it is bf16.
//
// 8-bit states.  A block of kStateBlock consecutive elements of a tensor
// shares one fp32 scale for m and one for r = sqrt(v): s = max |.| / 448,
// codes are the OCP float8 e4m3 nearest to m / s and to r / s.  The root
// halves the range that the second moment spans, so that e4m3's 17.8 octaves
// hold 35 of v; a positive r is never stored as zero (it is raised to the
// smallest positive code, 2^-9), since the update divides by it.  The update
// itself uses the unrounded m and v of this step.  A block whose state holds a
// NaN or an infinity gets the scale NaN: all of it reads as NaN.
//
// A wave owns whole blocks (four elements per lane), so a block's largest
// magnitude is one reduction within the wave and every element is read and
// written once.

#include <cmath>

#include "device_util.hpp"
#include "internal.hpp"

namespace sr {
namespace {

constexpr int kBlock = int(kStateBlock);
constexpr int kWaves = 4;
constexpr int kTensors = 80;       // per launch: the table travels in the kernel's arguments
constexpr float kTop = 448.0f;     // largest e4m3 value
constexpr float kTiny = 0.001953125f;  // smallest positive one, 2^-9

struct Tensor {
  void* param;
  const void* grad;
  int64_t n;
  int64_t state;  // first element of its states
};

struct AdamWParams {
  Tensor t[kTensors];
  uint32_t first[kTensors];  // first workgroup of each tensor
  uint8_t types[kTensors];   // bit 0: bf16 param, bit 1: bf16 grad
  int n_tensors;
  void* m;
  void* v;
  float* m_scale;  // null: fp32 states
  float* v_scale;
  const float* grad_scale;  // or null
  float b1, b2, one_b1, one_b2, decay, rate, inv_root_c2, eps;
};
static_assert(sizeof(AdamWParams) <= 4096, "kernel arguments");

// Four elements from element i of a tensor of n (zeros past its end).
__device__ __forceinline__ void load4(const void* p, bool bf16, int64_t i, int64_t n, float (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = 0.0f;
    if (i + j < n)
      x[j] = bf16 ? __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i + j]) << 16)
                  : static_cast<const float*>(p)[i + j];
  }
}

__device__ __forceinline__ void store4(void* p, bool bf16, int64_t i, int64_t n, const float (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (i + j < n) {
      if (bf16)
        static_cast<uint16_t*>(p)[i + j] = uint16_t(bf16_bits(x[j]));
      else
        static_cast<float*>(p)[i + j] = x[j];
    }
  }
}

__device__ __forceinline__ void decode4(uint32_t c, float s, float (&x)[4]) {
  x[0] = __builtin_amdgcn_cvt_f32_fp8(int(c), 0) * s;
  x[1] = __builtin_amdgcn_cvt_f32_fp8(int(c), 1) * s;
  x[2] = __builtin_amdgcn_cvt_f32_fp8(int(c), 2) * s;
  x[3] = __builtin_amdgcn_cvt_f32_fp8(int(c), 3) * s;
}

// Codes of a block, four elements per lane, and its scale.
template <bool kPositive>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], float* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b = abs_bits(x[j]);
    top = top > b ? top : b;
  }
  top = wave_max(top);
  if (top >= kF32InfBits) {
    *scale = __uint_as_float(0x7FC00000u);
    return 0;
  }
  const float s = __uint_as_float(top) / kTop;
  *scale = s;
  if (s == 0.0f) return 0;
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // A subnormal scale may have been rounded down: the clamp keeps its block's top a number.
    y[j] = fminf(fmaxf(x[j] / s, -kTop), kTop);
    if (kPositive) y[j] = x[j] > 0.0f ? fmaxf(y[j], kTiny) : 0.0f;
  }
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true));
}

__global__ __launch_bounds__(64 * kWaves) void adamw_kernel(const AdamWParams P) {
  int t = 0;  // the tensor of this workgroup: the last whose first workgroup is not past it
  for (int i = 1; i < P.n_tensors; ++i)
    if (P.first[i] <= blockIdx.x) t = i;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Tensor T = P.t[t];
  const bool p16 = P.types[t] & 1, g16 = P.types[t] & 2;
  const int64_t block = int64_t(blockIdx.x - P.first[t]) * kWaves + wave;
  if (block * kBlock >= T.n) return;
  const int64_t i = block * kBlock + lane * 4, n = T.n;
  float p[4], g[4], m[4], v[4];
  load4(T.param, p16, i, n, p);
  load4(T.grad, g16, i, n, g);
  const int64_t s0 = T.state + i;  // this lane's states; a multiple of 4
  const bool eight = P.m_scale != nullptr;
  const int64_t sb = T.state / kBlock + block;
  if (eight) {
    uint32_t cm = 0, cv = 0;
    cm = static_cast<const uint32_t*>(P.m)[s0 / 4];
    cv = static_cast<const uint32_t*>(P.v)[s0 / 4];
    decode4(cm, P.m_scale[sb], m);
    decode4(cv, P.v_scale[sb], v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= v[j];
  } else {
    load4(static_cast<const float*>(P.m) + T.state, false, i, n, m);
    load4(static_cast<const float*>(P.v) + T.state, false, i, n, v);
  }
  const float gs = P.grad_scale != nullptr ? *P.grad_scale : 1.0f;
  float root[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float gj = g[j] * gs;
    m[j] = P.b1 * m[j] + P.one_b1 * gj;
    v[j] = P.b2 * v[j] + P.one_b2 * (gj * gj);
    root[j] = sqrtf(v[j]);
    p[j] = p[j] * P.decay - P.rate * (m[j] / (root[j] * P.inv_root_c2 + P.eps));
  }
  store4(T.param, p16, i, n, p);
  if (eight) {
    // Elements past the tensor's end stay out of the block's scale and keep the code zero.
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j >= n) m[j] = root[j] = 0.0f;
    float ms, vs;
    const uint32_t cm = encode4<false>(m, &ms), cv = encode4<true>(root, &vs);
    static_cast<uint32_t*>(P.m)[s0 / 4] = cm;
    static_cast<uint32_t*>(P.v)[s0 / 4] = cv;
    if (lane == 0) {
      P.m_scale[sb] = ms;
      P.v_scale[sb] = vs;
    }
  } else {
    store4(static_cast<float*>(P.m) + T.state, false, i, n, m);
    store4(static_cast<float*>(P.v) + T.state, false, i, n, v);
  }
}

}  // namespace

sr_status launch_adamw(const AdamWRequest& rq) {
  AdamWParams P{};
  P.m = rq.m;
  P.v = rq.v;
  P.m_scale = rq.m_scale;
  P.v_scale = rq.v_scale;
  P.grad_scale = rq.grad_scale;
  P.b1 = float(rq.beta1);
  P.b2 = float(rq.beta2);
  P.one_b1 = float(1.0 - rq.beta1);
  P.one_b2 = float(1.0 - rq.beta2);
  P.decay = float(1.0 - rq.lr * rq.weight_decay);
  P.rate = float(rq.lr / (1.0 - std::pow(rq.beta1, double(rq.step))));
  P.inv_root_c2 = float(1.0 / std::sqrt(1.0 - std::pow(rq.beta2, double(rq.step))));
  P.eps = float(rq.eps);
  // Fills tables of up to kTensors tensors; the first pass only checks that
  // every launch's grid fits.
  for (int pass = 0; pass < 2; ++pass) {
    int64_t state = 0, blocks = 0;
    P.n_tensors = 0;
    for (int64_t i = 0; i <= rq.n_tensors; ++i) {
      if (P.n_tensors > 0 && (i == rq.n_tensors || P.n_tensors == kTensors)) {
        if (blocks > kMaxBlocks256)
          return fail(SR_ERR_UNSUPPORTED, "%lld elements exceed one launch's grid",
                      (long long)(blocks * kWaves * kBlock));
        if (pass == 1) {
          hipLaunchKernelGGL(adamw_kernel, dim3(uint32_t(blocks)), dim3(64 * kWaves), 0, rq.stream, P);
          const hipError_t err = hipGetLastError();
          if (err != hipSuccess) return fail(SR_ERR_HIP, "AdamW launch: %s", hipGetErrorString(err));
        }
        P.n_tensors = 0;
        blocks = 0;
      }
      if (i == rq.n_tensors) break;
      const sr_adamw_tensor& t = rq.tensors[i];
      if (t.n > 0 && t.grad != nullptr) {
        const int k = P.n_tensors++;
        P.t[k] = Tensor{t.param, t.grad, t.n, state};
        P.first[k] = uint32_t(blocks);
        P.types[k] = uint8_t((t.param_dtype == SR_BF16 ? 1 : 0) | (t.grad_dtype == SR_BF16 ? 2 : 0));
        blocks += (t.n + kWaves * kBlock - 1) / (kWaves * kBlock);
      }
      state += adamw_span(t.n);
    }
  }
  return SR_OK;
}

}  // namespace sr
