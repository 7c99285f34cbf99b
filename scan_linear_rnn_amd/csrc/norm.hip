// Root-mean-square norm of rows, with the residual's addition in front:
//
//     t = x + r  (stored in r's type),   y = t / sqrt(mean(t^2) + eps) * w
//
// y in x's type, or as 8-bit codes with a scale per row (quant.hip's), made of the
// fp32 values; and its backward pass,
//
//     n = t / rms,  g = dy w,  dx = (g - n mean(g n)) / rms + dt,  dw = sum over rows of dy n
//
// Bound by the rows' bytes: a row is read once and stays in registers, 8 elements
// per lane at a time; a row has 16 lanes, 32, a wave or several, by its length.  Sum and
// 8-bit codes of 131072 x 2048 in bf16 take 329 us (5.7 TB/s); the backward pass of 16384 x
// 2048 with fp32 sums 82 us and 5 for the weight's gradient (5.7 TB/s).

#include "layer_util.hpp"
#include "quant.hpp"

namespace sr {
namespace {

constexpr int kV = 8;  // elements per lane and chunk

struct None {};  // no residual

// A lane's chunks of a row of D elements, `step` apart from c0 on; zeros behind the row.  kWhole: D is
// a multiple of a chunk, and all loads are on the way before the first is waited for.
template <bool kWhole, int NV, typename T>
__device__ __forceinline__ void load_row(const T* row, int c0, int step, int D, float (&v)[NV][kV]) {
  if constexpr (kWhole) {
    Raw<T, kV> raw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = c0 + j * step;
      load_raw<true>(row + (c < D ? c : 0), kV, raw[j]);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      values(raw[j], v[j]);
      if (c0 + j * step >= D) {
#pragma unroll
        for (int e = 0; e < kV; ++e) v[j][e] = 0.0f;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) load_some(row + c0 + j * step, D - c0 - j * step, v[j]);
  }
}

// Sum, or largest value, over a row of LPR lanes and WPR waves, in all of them;
// the waves' values meet in LDS (two barriers).
template <int LPR, int WPR, typename V, typename Join>
__device__ __forceinline__ V row_all(V v, V* s, Join join) {
#pragma unroll
  for (int m = 1; m < LPR; m *= 2) v = join(v, V(__shfl_xor(v, m)));
  if constexpr (WPR > 1) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int k = 1; k < WPR; ++k) v = join(v, s[k]);
  }
  return v;
}
template <int LPR, int WPR>
__device__ __forceinline__ float row_sum(float v, float* s) {
  return row_all<LPR, WPR>(v, s, [](float a, float b) { return a + b; });
}

// LPR lanes and WPR waves per row (LPR < 64 only with one wave), NV chunks per
// lane.  X: the type of x and y, R: of the residual and the sum (None: there
// is none); CODES: 8-bit codes instead of y.
template <typename X, typename R, int LPR, int WPR, int NV, bool CODES, bool kWhole>
__global__ __launch_bounds__(WPR > 4 ? WPR * 64 : 256) void norm_kernel(const NormRequest P) {
  constexpr int kThreads = WPR > 4 ? WPR * 64 : 256;
  constexpr int kRows = kThreads / (LPR * WPR);
  constexpr bool kResidual = !std::is_same_v<R, None>;
  __shared__ float s_all[WPR];
  __shared__ uint32_t s_top[WPR];
  const int c0 = threadIdx.x % (LPR * WPR) * kV;
  const int D = int(P.D);
  float w[NV][kV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = c0 + j * LPR * WPR * kV;
    if (P.w_dtype == SR_BF16)
      load_some(static_cast<const uint16_t*>(P.w) + c, D - c, w[j]);
    else
      load_some(static_cast<const float*>(P.w) + c, D - c, w[j]);
  }
  const int64_t last = P.M - 1;
  for (int64_t block = blockIdx.x; block * kRows < P.M; block += gridDim.x) {
    const int64_t want = block * kRows + threadIdx.x / (LPR * WPR);
    const bool live = want < P.M;
    const int64_t row = live ? want : last;
    float t[NV][kV];
    float sum = 0.0f;
    load_row<kWhole>(static_cast<const X*>(P.x) + row * P.ld_x, c0, LPR * WPR * kV, D, t);
    if constexpr (kResidual) {
      float r[NV][kV];
      load_row<kWhole>(static_cast<const R*>(P.r) + row * P.ld_r, c0, LPR * WPR * kV, D, r);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * LPR * WPR * kV;
#pragma unroll
        for (int e = 0; e < kV; ++e) t[j][e] = to_f32(from_f32<R>(t[j][e] + r[j][e]));
        if (live) store_some(static_cast<R*>(P.total) + row * P.D + c, D - c, t[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < kV; ++e) sum = fmaf(t[j][e], t[j][e], sum);
    sum = row_sum<LPR, WPR>(sum, s_all);
    const float inv = 1.0f / sqrtf(sum / float(D) + P.eps);
    if constexpr (!CODES) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * LPR * WPR * kV;
#pragma unroll
        for (int e = 0; e < kV; ++e) t[j][e] = t[j][e] * inv * w[j][e];
        if (live) store_some(static_cast<X*>(P.y) + row * P.D + c, D - c, t[j]);
      }
    } else {
      uint32_t bits = 0;  // of the largest magnitude: infinities and NaNs on top
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < kV; ++e) {
          t[j][e] = t[j][e] * inv * w[j][e];
          const uint32_t b = abs_bits(t[j][e]);
          bits = bits > b ? bits : b;
        }
      bits = row_all<LPR, WPR>(bits, s_top, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
      const float s = row_scale(bits);
      const bool plain = divides_plainly(s);
      const float r = plain ? __fdiv_rn(1.0f, s) : 0.0f;
      if (live && c0 == 0) P.scale[row] = s;
      int8_t* dst = P.q + row * P.ld_q;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = c0 + j * LPR * WPR * kV;
        u32x2 out{};
#pragma unroll
        for (int e = 0; e < kV; ++e) {
          const uint32_t q = plain ? uint32_t(int(rintf(divided(t[j][e], s, r)))) & 0xFFu : code(t[j][e], s, s > 0.0f);
          out[e / 4] |= q << (8 * (e % 4));
        }
        if (live && c < P.ld_q) *reinterpret_cast<u32x2*>(dst + c) = out;  // zeros behind the row
      }
    }
  }
}

template <typename X, typename R, int LPR, int WPR, int NV, bool kWhole>
__global__ __launch_bounds__(WPR > 4 ? WPR * 64 : 256) void norm_backward_kernel(const NormRequest P) {
  constexpr int kThreads = WPR > 4 ? WPR * 64 : 256;
  constexpr int kRows = kThreads / (LPR * WPR);
  __shared__ float s_all[WPR];
  __shared__ float s_dw[kRows > 1 ? LPR * NV * kV : 1];
  const int c0 = threadIdx.x % (LPR * WPR) * kV;
  const int D = int(P.D);
  float w[NV][kV], dw[NV][kV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = c0 + j * LPR * WPR * kV;
    if (P.w_dtype == SR_BF16)
      load_some(static_cast<const uint16_t*>(P.w) + c, D - c, w[j]);
    else
      load_some(static_cast<const float*>(P.w) + c, D - c, w[j]);
#pragma unroll
    for (int e = 0; e < kV; ++e) dw[j][e] = 0.0f;
  }
  for (int64_t block = blockIdx.x; block * kRows < P.M; block += gridDim.x) {
    const int64_t want = block * kRows + threadIdx.x / (LPR * WPR);
    const bool live = want < P.M;
    const int64_t row = live ? want : P.M - 1;
    float t[NV][kV], g[NV][kV], dt[NV][kV];
    float square = 0.0f, cross = 0.0f;  // of t, and of g t
    load_row<kWhole>(static_cast<const R*>(P.t) + row * P.ld_t, c0, LPR * WPR * kV, D, t);
    load_row<kWhole>(static_cast<const X*>(P.dy) + row * P.ld_dy, c0, LPR * WPR * kV, D, g);
    if (P.dt) {
      load_row<kWhole>(static_cast<const R*>(P.dt) + row * P.ld_dt, c0, LPR * WPR * kV, D, dt);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < kV; ++e) dt[j][e] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        square = fmaf(t[j][e], t[j][e], square);
        cross = fmaf(g[j][e] * w[j][e], t[j][e], cross);
      }
    square = row_sum<LPR, WPR>(square, s_all);
    cross = row_sum<LPR, WPR>(cross, s_all);
    const float inv = 1.0f / sqrtf(square / float(D) + P.eps);
    const float mean = cross * inv / float(D);  // of g n
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = c0 + j * LPR * WPR * kV;
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        const float n = t[j][e] * inv;
        if (live) dw[j][e] = fmaf(g[j][e], n, dw[j][e]);
        t[j][e] = fmaf(fmaf(-n, mean, g[j][e] * w[j][e]), inv, dt[j][e]);
      }
      if (live) store_some(static_cast<R*>(P.dx) + row * P.D + c, D - c, t[j]);
    }
  }
  // The workgroup's rows at once add up theirs in turn.
  float* to = P.parts + int64_t(blockIdx.x) * P.D;
  if constexpr (kRows > 1) {
#pragma unroll 1
    for (int k = 0; k < kRows; ++k) {
      if (int(threadIdx.x) / LPR == k) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            const int c = c0 + j * LPR * kV + e;
            s_dw[c] = k == 0 ? dw[j][e] : s_dw[c] + dw[j][e];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < D; c += kThreads) to[c] = s_dw[c];
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = c0 + j * LPR * WPR * kV;
      store_some(to + c, D - c, dw[j]);
    }
  }
}

__global__ __launch_bounds__(1024) void norm_sums_kernel(const float* parts, int64_t rows, int64_t D, float* dw) {
  column_sums(parts, rows, D, [&](int64_t c, float sum) { dw[c] = sum; });
}

template <int LPR, int WPR, int NV>
struct Shape {
  static constexpr int kLanes = LPR, kWaves = WPR, kChunks = NV;
  static constexpr int kThreads = WPR > 4 ? WPR * 64 : 256;
  static constexpr int kRows = kThreads / (LPR * WPR);
};
// Calls f with the lanes, waves and chunks per lane for rows of D elements (for codes:
// the padded row): as few lanes as hold a row in one or two chunks each, so that no lane
// idles and the reductions are short, and four waves from 1024 elements on.  Measured in us,
// bf16, one wave / four: codes of 131072 x 2048 346 / 337, of 256 x 2048 6.5 / 4.1; fp32 sums:
// codes of 131072 x 2048 559 / 516, their backward 575 / 548, of 256 rows 12.1 / 7.1; 131072 x 1024
// codes 173 / 271.  Four waves of four chunks / of two, 65536 x 4096: codes 458 / 336, backward with
// fp32 sums 614 / 521.  Up to 8192 the forward kernels are faster with eight waves of two chunks than
// with four of four (32768 rows of codes 348 / 336, 1024 rows 16.2 / 14.3), the backward kernel is
// not (563 / 526).
template <bool kBackward, typename F>
void by_width(int64_t D, F f) {
  if (D <= 16 * kV) return f(Shape<16, 1, 1>{});
  if (D <= 32 * kV) return f(Shape<32, 1, 1>{});
  if (D <= 64 * kV) return f(Shape<64, 1, 1>{});
  if (D <= 2 * 64 * kV) return f(Shape<64, 1, 2>{});
  if (D <= 256 * kV) return f(Shape<64, 4, 1>{});
  if (D <= 2 * 256 * kV) return f(Shape<64, 4, 2>{});
  if (D <= 4 * 256 * kV) return f(Shape<64, kBackward ? 4 : 8, kBackward ? 4 : 2>{});
  return f(Shape<64, 8, 4>{});
}

// Workgroups.  Forward: one for its few rows, and no loop in it, is faster than as many as the CUs
// hold, each with its share of the rows (the loop's stores are in the way of the next row's loads):
// 1024 / 8192 / one each, us: 131072 x 2048 codes 373 / 406 / 337, 1048576 x 128 198 / 188 / 168, but
// 16384 x 16384 384 / 431 / 431, whose workgroups fill half of a CU.  The backward kernel writes its
// sums for the weight once per workgroup: with 256 / 512 / 1024 of them 131072 x 2048 takes 951 / 548 /
// 564, 8192 x 4096 90 / 72 / 79, 1024 x 16384 50 / 57 / 70, 65536 x 512 70 / 44 / 36.
template <typename S>
constexpr int64_t kForwardBlocks = S::kWaves * S::kChunks == 32 ? 1024 : 1 << 20;
template <typename S>
constexpr int64_t kBackwardBlocks = S::kWaves == 1 ? 1024 : S::kWaves == 4 ? 512 : 256;

sr_status launched(const char* what) {
  const hipError_t err = hipGetLastError();
  return err == hipSuccess ? SR_OK : fail(SR_ERR_HIP, "%s: %s", what, hipGetErrorString(err));
}

int64_t capped(int64_t blocks, int64_t most) { return blocks < most ? blocks : most; }

template <typename X, typename R>
void launch_forward(const NormRequest& P) {
  by_width<false>(P.q ? P.ld_q : P.D, [&](auto shape) {
    using S = decltype(shape);
    const int64_t blocks = capped((P.M + S::kRows - 1) / S::kRows, kForwardBlocks<S>);
    auto run = [&](auto* whole, auto* any) {
      hipLaunchKernelGGL(P.D % kV == 0 ? whole : any, dim3(uint32_t(blocks)), dim3(S::kThreads), 0, P.stream, P);
    };
    if (P.q)
      run(norm_kernel<X, R, S::kLanes, S::kWaves, S::kChunks, true, true>,
          norm_kernel<X, R, S::kLanes, S::kWaves, S::kChunks, true, false>);
    else
      run(norm_kernel<X, R, S::kLanes, S::kWaves, S::kChunks, false, true>,
          norm_kernel<X, R, S::kLanes, S::kWaves, S::kChunks, false, false>);
  });
}

template <typename X, typename R>
void launch_back(const NormRequest& P) {
  by_width<true>(P.D, [&](auto shape) {
    using S = decltype(shape);
    auto run = [&](auto* kernel) {
      hipLaunchKernelGGL(kernel, dim3(uint32_t(norm_backward_blocks(P.M, P.D))), dim3(S::kThreads), 0, P.stream, P);
    };
    if (P.D % kV == 0)
      run(norm_backward_kernel<X, R, S::kLanes, S::kWaves, S::kChunks, true>);
    else
      run(norm_backward_kernel<X, R, S::kLanes, S::kWaves, S::kChunks, false>);
  });
}

}  // namespace

int64_t norm_backward_blocks(int64_t M, int64_t D) {
  int64_t blocks = 0;
  by_width<true>(D, [&](auto shape) {
    using S = decltype(shape);
    blocks = capped((M + S::kRows - 1) / S::kRows, kBackwardBlocks<S>);
  });
  return blocks;
}

sr_status launch_norm(const NormRequest& P) {
  const bool x16 = P.dtype == SR_BF16, r16 = P.r_dtype == SR_BF16;
  if (!P.r)
    x16 ? launch_forward<uint16_t, None>(P) : launch_forward<float, None>(P);
  else if (r16)
    x16 ? launch_forward<uint16_t, uint16_t>(P) : launch_forward<float, uint16_t>(P);
  else
    x16 ? launch_forward<uint16_t, float>(P) : launch_forward<float, float>(P);
  return launched("norm");
}

sr_status launch_norm_backward(const NormRequest& P) {
  const bool x16 = P.dtype == SR_BF16, r16 = P.r_dtype == SR_BF16;
  if (P.M > 0) {
    if (r16)
      x16 ? launch_back<uint16_t, uint16_t>(P) : launch_back<float, uint16_t>(P);
    else
      x16 ? launch_back<uint16_t, float>(P) : launch_back<float, float>(P);
  }
  sr_status st = launched("norm backward");
  if (st != SR_OK) return st;
  hipLaunchKernelGGL(norm_sums_kernel, dim3(uint32_t((P.D + 63) / 64)), dim3(1024), 0, P.stream, P.parts,
                     norm_backward_blocks(P.M, P.D), P.D, P.dw);
  return launched("norm gradient sums");
}

}  // namespace sr
