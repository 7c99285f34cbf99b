// One AdamW step over many tensors in few launches, states in fp32 or in 8
// bits.  For each element, with the number t of its tensor's step and
// c1 = 1 - b1^t, c2 = 1 - b2^t:
//
//     g = grad * grad_scale
//     m = b1 m + (1 - b1) g        v = b2 v + (1 - b2) g^2
//     p = p (1 - lr wd) - (lr / c1) m / (sqrt(v) / sqrt(c2) + eps)
//
// in fp32 whatever the tensors' types; p is rounded once when it is bf16.
//
// 8-bit states.  A block of kStateBlock consecutive elements of a tensor
// shares one fp32 scale for m and one for r = sqrt(v): s = max |.| / 448 (times
// the fp32 nearest to 1 / 448), codes are the OCP float8 e4m3 nearest to m / s
// and to r / s.  The root
// halves the range that the second moment spans, so that e4m3's 17.8 octaves
// hold 35 of v; a positive r is never stored as zero (it is raised to the
// smallest positive code, 2^-9), since the update divides by it.  The update
// itself uses the unrounded m and v of this step.  Codes of r lie 6 to 12%
// apart and one step moves r by less, so over many steps an element follows its
// block's largest one, held exactly, and not a change of its own gradients (the
// header says how far that goes).  A block whose state holds a
// NaN or an infinity gets the scale NaN: all of it reads as NaN.
//
// A wave owns whole blocks (four elements per lane), so a block's largest
// magnitude is one reduction within the wave and every element is read and
// written once.  The step is bound by those bytes (28 per element in fp32, 14
// with bf16 gradients and 8-bit states): four blocks per wave keep 16 loads
// in flight, and the table of tensors travels in the kernel's arguments, so
// that a call is one launch for every 64 tensors and nothing is copied.
// Measured (100.7 M fp32 parameters): fp32 states 465 us, 6.05 TB/s; bf16
// gradients and 8-bit states 242 us, 5.8 TB/s.

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "device_util.hpp"
#include "internal.hpp"

namespace sr {
namespace {

constexpr int kBlock = int(kStateBlock);
constexpr int kWaves = 4;
constexpr int kBlocks = 4;         // per wave
constexpr int kTensors = 64;       // per launch: one lane each finds a workgroup's tensor
// Tensors up to this long take one block per wave: their ends go block by
// block, each at a load's latency.  Measured (us, one block / four, 8-bit states):
// 60 tensors of 4096 elements 5.1 / 7.0, 49 of 1 to 73728 4.9 / 7.9; 60 of 65536
// 18.0 / 14.6.
constexpr int64_t kShort = 16384;
constexpr float kTop = 448.0f;     // largest e4m3 value
constexpr float kTiny = 0.001953125f;  // smallest positive one, 2^-9

struct Tensor {
  void* param;
  const void* grad;
  int64_t n;
  int64_t state;  // first element of its states
};

// What a tensor's step number makes of the rate and of the root: lr / c1, 1 / sqrt(c2).
struct Correction {
  float rate, inv_root_c2;
};

struct AdamWParams {
  Tensor t[kTensors];
  uint32_t first[kTensors];  // first workgroup of each tensor; past the last: none
  uint32_t types[kTensors];  // bit 0: bf16 param, bit 1: bf16 grad, bit 2: aligned for vector accesses, bit 3: short
  Correction bias[kTensors];
  void* m;
  void* v;
  float* m_scale;  // null: fp32 states
  float* v_scale;
  const float* grad_scale;  // or null
  float b1, b2, one_b1, one_b2, decay, eps;
};
static_assert(sizeof(AdamWParams) <= 4096, "kernel arguments");

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// Four elements from element i: 16 bytes of fp32 or 8 of bf16.
template <bool kBF16>
__device__ __forceinline__ f32x4 load4(const void* p, int64_t i) {
  if constexpr (kBF16) {
    const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + i));
    return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                 __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u)};
  } else {
    return __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i));
  }
}
template <bool kBF16>
__device__ __forceinline__ void store4(void* p, int64_t i, f32x4 x) {
  if constexpr (kBF16) {
    u32x2 w;
    w.x = bf16_pair(x[0], x[1]);
    w.y = bf16_pair(x[2], x[3]);
    __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p) + i));
  } else {
    __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(static_cast<float*>(p) + i));
  }
}

// The same one element at a time, for a tensor's last elements and for
// pointers at odd elements (zeros past n).
__device__ __forceinline__ f32x4 load4_any(const void* p, bool bf16, int64_t i, int64_t n) {
  f32x4 x{};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n)
      x[j] = bf16 ? __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i + j]) << 16)
                  : static_cast<const float*>(p)[i + j];
  return x;
}
__device__ __forceinline__ void store4_any(void* p, bool bf16, int64_t i, int64_t n, f32x4 x) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (i + j < n) {
      if (bf16)
        static_cast<uint16_t*>(p)[i + j] = uint16_t(bf16_pair(x[j], 0.0f));
      else
        static_cast<float*>(p)[i + j] = x[j];
    }
  }
}

__device__ __forceinline__ f32x4 decode4(uint32_t c, float s) {
  return f32x4{__builtin_amdgcn_cvt_f32_fp8(int(c), 0), __builtin_amdgcn_cvt_f32_fp8(int(c), 1),
               __builtin_amdgcn_cvt_f32_fp8(int(c), 2), __builtin_amdgcn_cvt_f32_fp8(int(c), 3)} * s;
}

// Codes of a block, four elements per lane, and its scale (uniform).
template <bool kPositive>
__device__ __forceinline__ uint32_t encode4(f32x4 x, float* scale) {
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
  const float s = __uint_as_float(top) * (1.0f / kTop);
  *scale = s;
  if (s == 0.0f) return 0;
  const bool plain = divides_plainly(s);
  const float inv = plain ? __fdiv_rn(1.0f, s) : 0.0f;
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // A subnormal scale may have been rounded down: the clamp keeps its block's top a number.
    const float q = plain ? divided(x[j], s, inv) : __fdiv_rn(x[j], s);
    y[j] = kPositive ? (x[j] > 0.0f ? __builtin_amdgcn_fmed3f(q, kTiny, kTop) : 0.0f)
                     : __builtin_amdgcn_fmed3f(q, -kTop, kTop);
  }
  const int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true));
}

// One element: p, m and v after the step, and r = sqrt(v).  What becomes a
// state is rounded operation by operation, as written, never fused, and the
// root is the IEEE one: where an element lies on the tie of two 8-bit codes,
// the code is then a function of the formula and not of what the compiler
// contracts.  The reciprocal in p's update is good to an ulp, 2^-23 of it.
__device__ __forceinline__ void update(const AdamWParams& P, Correction c, float g, float& p, float& m, float& v,
                                       float& r) {
#pragma clang fp contract(off)
  m = m * P.b1 + g * P.one_b1;
  v = v * P.b2 + g * g * P.one_b2;
  r = sqrtf(v);
  p = p * P.decay - c.rate * (m * __builtin_amdgcn_rcpf(r * c.inv_root_c2 + P.eps));
}

// The states of a block, as loaded: fp32, or codes and scales.
template <bool kEight>
struct RawStates;
template <>
struct RawStates<false> {
  f32x4 m, v;
  __device__ __forceinline__ void load(const AdamWParams& P, int64_t at, int64_t) {
    m = load4<false>(P.m, at);
    v = load4<false>(P.v, at);
  }
  __device__ __forceinline__ void get(f32x4& mo, f32x4& vo) const { mo = m; vo = v; }
  static __device__ __forceinline__ void store(const AdamWParams& P, int64_t at, int64_t, f32x4 m, f32x4 v, f32x4) {
    store4<false>(P.m, at, m);
    store4<false>(P.v, at, v);
  }
};
template <>
struct RawStates<true> {
  uint32_t m, v;
  float ms, vs;
  __device__ __forceinline__ void load(const AdamWParams& P, int64_t at, int64_t block) {
    m = __builtin_nontemporal_load(static_cast<const uint32_t*>(P.m) + at / 4);
    v = __builtin_nontemporal_load(static_cast<const uint32_t*>(P.v) + at / 4);
    ms = P.m_scale[block];
    vs = P.v_scale[block];
  }
  __device__ __forceinline__ void get(f32x4& mo, f32x4& vo) const {
    mo = decode4(m, ms);
    vo = decode4(v, vs);
    vo *= vo;
  }
  static __device__ __forceinline__ void store(const AdamWParams& P, int64_t at, int64_t block, f32x4 m, f32x4,
                                               f32x4 r) {
    float ms, vs;
    const uint32_t cm = encode4<false>(m, &ms), cv = encode4<true>(r, &vs);
    __builtin_nontemporal_store(cm, static_cast<uint32_t*>(P.m) + at / 4);
    __builtin_nontemporal_store(cv, static_cast<uint32_t*>(P.v) + at / 4);
    if ((threadIdx.x & 63) == 0) {
      P.m_scale[block] = ms;
      P.v_scale[block] = vs;
    }
  }
};

// kBlocks whole blocks of an aligned tensor, from block0 in steps of kWaves.
template <bool kEight, bool kP16, bool kG16>
__device__ __forceinline__ void run_blocks(const AdamWParams& P, const Tensor& T, Correction c, int64_t block0,
                                           float gs) {
  const int lane = threadIdx.x & 63;
  f32x4 p[kBlocks], g[kBlocks];
  RawStates<kEight> s[kBlocks];
#pragma unroll
  for (int u = 0; u < kBlocks; ++u) {
    const int64_t i = (block0 + u * kWaves) * kBlock + lane * 4;
    p[u] = load4<kP16>(T.param, i);
    g[u] = load4<kG16>(T.grad, i);
    s[u].load(P, T.state + i, T.state / kBlock + block0 + u * kWaves);
  }
#pragma unroll
  for (int u = 0; u < kBlocks; ++u) {
    const int64_t i = (block0 + u * kWaves) * kBlock + lane * 4;
    f32x4 m, v, r;
    s[u].get(m, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float pj = p[u][j], mj = m[j], vj = v[j], rj;
      update(P, c, g[u][j] * gs, pj, mj, vj, rj);
      p[u][j] = pj;
      m[j] = mj;
      v[j] = vj;
      r[j] = rj;
    }
    store4<kP16>(T.param, i, p[u]);
    RawStates<kEight>::store(P, T.state + i, T.state / kBlock + block0 + u * kWaves, m, v, r);
  }
}

// One block that ends the tensor, or of one that is not aligned.
template <bool kEight>
__device__ __forceinline__ void run_any(const AdamWParams& P, const Tensor& T, Correction c, bool p16, bool g16,
                                        int64_t block, float gs) {
  const int64_t i = block * kBlock + (threadIdx.x & 63) * 4, n = T.n;
  f32x4 p = load4_any(T.param, p16, i, n);
  const f32x4 g = load4_any(T.grad, g16, i, n);
  RawStates<kEight> s;
  s.load(P, T.state + i, T.state / kBlock + block);  // a tensor's span holds whole blocks
  f32x4 m, v, r;
  s.get(m, v);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float pj = p[j], mj = m[j], vj = v[j], rj;
    update(P, c, g[j] * gs, pj, mj, vj, rj);
    const bool on = i + j < n;  // the span's tail keeps out of the block's scale, and stays zero
    p[j] = pj;
    m[j] = on ? mj : 0.0f;
    v[j] = on ? vj : 0.0f;
    r[j] = on ? rj : 0.0f;
  }
  store4_any(T.param, p16, i, n, p);
  RawStates<kEight>::store(P, T.state + i, T.state / kBlock + block, m, v, r);
}

template <bool kEight>
__global__ __launch_bounds__(64 * kWaves) void adamw_kernel(const AdamWParams P) {
  const int lane = threadIdx.x & 63;
  // The tensor of this workgroup: the last whose first workgroup is not past it.
  const int t = __builtin_popcountll(__builtin_amdgcn_ballot_w64(P.first[lane] <= blockIdx.x)) - 1;
  const Tensor T = P.t[t];
  const uint32_t types = P.types[t];
  const Correction bias = P.bias[t];
  const float gs = P.grad_scale != nullptr ? *P.grad_scale : 1.0f;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = types & 8 ? 1 : kBlocks;
  const int64_t first = int64_t(blockIdx.x - P.first[t]) * (kWaves * blocks), block0 = first + wave;
  if (blocks == kBlocks && (first + kWaves * kBlocks) * kBlock <= T.n && (types & 4)) {
    switch (types & 3) {
      case 0: return run_blocks<kEight, false, false>(P, T, bias, block0, gs);
      case 1: return run_blocks<kEight, true, false>(P, T, bias, block0, gs);
      case 2: return run_blocks<kEight, false, true>(P, T, bias, block0, gs);
      default: return run_blocks<kEight, true, true>(P, T, bias, block0, gs);
    }
  }
#pragma unroll 1
  for (int u = 0; u < blocks; ++u)
    if ((block0 + u * kWaves) * kBlock < T.n)
      run_any<kEight>(P, T, bias, types & 1, types & 2, block0 + u * kWaves, gs);
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool takes_part(const sr_adamw_tensor& t) { return t.n > 0 && t.grad != nullptr; }

// Workgroups of different tensors run in any order: no two tensors of a step
// may share memory.  The host sorts their ranges (those that are in order already
// are only looked through): 0.2 us of a call over 49 tensors (8.6 -> 8.8 us).
sr_status check_disjoint(int64_t n_tensors, const sr_adamw_tensor* tensors) {
  struct Range {
    uintptr_t begin, end;
  };
  constexpr int64_t kOnStack = 256;
  Range few[kOnStack];
  std::unique_ptr<Range[]> many;
  if (n_tensors > kOnStack) {
    many.reset(new (std::nothrow) Range[size_t(n_tensors)]);
    if (!many) return fail(SR_ERR_UNSUPPORTED, "no host memory for %lld tensors", (long long)n_tensors);
  }
  Range* r = many ? many.get() : few;
  size_t n = 0;
  bool ascending = true;
  for (int64_t i = 0; i < n_tensors; ++i) {
    if (!takes_part(tensors[i])) continue;
    const uintptr_t at = reinterpret_cast<uintptr_t>(tensors[i].param);
    r[n] = Range{at, at + uintptr_t(tensors[i].n) * (tensors[i].param_dtype == SR_BF16 ? 2 : 4)};
    ascending = ascending && (n == 0 || r[n - 1].begin <= at);
    ++n;
  }
  if (!ascending) std::sort(r, r + n, [](const Range& a, const Range& b) { return a.begin < b.begin; });
  for (size_t i = 1; i < n; ++i)
    if (r[i].begin < r[i - 1].end)
      return fail(SR_ERR_INVALID_ARGUMENT, "two tensors of the step share memory (a parameter given twice?)");
  return SR_OK;
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
  P.eps = float(rq.eps);
  int64_t step = 0;  // the one that bias belongs to: neighbours mostly share it
  Correction bias{};
  // Fills tables of up to kTensors tensors; the first pass only checks that
  // every launch's grid fits.
  constexpr int64_t kPer = int64_t(kWaves) * kBlocks * kBlock;  // elements of a workgroup
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1) {
      const sr_status st = check_disjoint(rq.n_tensors, rq.tensors);
      if (st != SR_OK) return st;
    }
    int64_t state = 0, blocks = 0;
    int k = 0;  // tensors in the table
    for (int64_t i = 0; i <= rq.n_tensors; ++i) {
      if (k > 0 && (i == rq.n_tensors || k == kTensors)) {
        if (blocks > kMaxBlocks256)
          return fail(SR_ERR_UNSUPPORTED, "%lld elements exceed one launch's grid", (long long)(blocks * kPer));
        if (pass == 1) {
          for (; k < kTensors; ++k) P.first[k] = UINT32_MAX;
          if (rq.m_scale != nullptr)
            hipLaunchKernelGGL(adamw_kernel<true>, dim3(uint32_t(blocks)), dim3(64 * kWaves), 0, rq.stream, P);
          else
            hipLaunchKernelGGL(adamw_kernel<false>, dim3(uint32_t(blocks)), dim3(64 * kWaves), 0, rq.stream, P);
          const hipError_t err = hipGetLastError();
          if (err != hipSuccess) return fail(SR_ERR_HIP, "AdamW launch: %s", hipGetErrorString(err));
        }
        k = 0;
        blocks = 0;
      }
      if (i == rq.n_tensors) break;
      const sr_adamw_tensor& t = rq.tensors[i];
      if (takes_part(t)) {
        const bool p16 = t.param_dtype == SR_BF16, g16 = t.grad_dtype == SR_BF16;
        const bool wide = aligned(t.param, p16 ? 8 : 16) && aligned(t.grad, g16 ? 8 : 16);
        P.t[k] = Tensor{t.param, t.grad, t.n, state};
        P.first[k] = uint32_t(blocks);
        const int64_t now = rq.steps != nullptr ? rq.steps[i] : rq.step;
        if (now != step) {
          step = now;
          bias.rate = float(rq.lr / (1.0 - std::pow(rq.beta1, double(now))));
          bias.inv_root_c2 = float(1.0 / std::sqrt(1.0 - std::pow(rq.beta2, double(now))));
        }
        P.bias[k] = bias;
        const bool brief = t.n <= kShort;
        P.types[k] = uint32_t((p16 ? 1 : 0) | (g16 ? 2 : 0) | (wide ? 4 : 0) | (brief ? 8 : 0));
        const int64_t per = brief ? kPer / kBlocks : kPer;
        blocks += (t.n + per - 1) / per;
        ++k;
      }
      state += adamw_span(t.n);
    }
  }
  return SR_OK;
}

}  // namespace sr
