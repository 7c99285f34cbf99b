// Backward pass of the selective scan (selective.hip has the forward and the
// notation).  With s the output before the gate, ds = dy silu(z) and
// a_n = exp(dt A_n), backwards over the tokens:
//
//     G_n  <- G_n + ds C_n                      (dC_n = sum over channels of ds h_n)
//     dB_n  = sum over channels of G_n dt u
//     du    = dt sum_n G_n B_n + skip ds
//     q_n   = a_n G_n h_n(t-1)
//     ddt   = u sum_n G_n B_n + sum_n A_n q_n,  dA_n += dt q_n
//     G_n  <- a_n G_n
//     ddelta = ddt sigma(delta + bias),  dz = dy s silu'(z)
//
// The states are computed again from marks: the forward's first pass
// (scan_kernel with kStates) writes what each chunk has made of a zero state in front of
// every 16 tokens, and the sum of its steps there, so that the state itself is one
// exponential and one product away from the chunk's start.  A workgroup then owns
// 64 channels of one chunk, a lane each, goes back over its tiles of 16
// tokens, runs each forward into registers and back again.  The sums over
// channels, dB and dC, are 64 values per wave and tile (16 tokens, 4 states) to be
// summed over 64 lanes: a halving exchange (swaps of half waves, then of rows,
// then DPP) leaves one sum in every lane at about two instructions per value,
// where separate sums would take six.  They go out per 64 channels and
// reduce_kernel adds those up, always in the same order.

#include "layer_util.hpp"

namespace sr {
namespace {

template <int kCtrl>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(
      uint32_t(__builtin_amdgcn_mov_dpp(int(__float_as_uint(x)), kCtrl, 0xF, 0xF, true)));
}

// Sums of 64 values over the 64 lanes: lane l returns the sum of v[l].
__device__ __forceinline__ float sum64(float (&v)[64], int lane) {
#pragma unroll
  for (int k = 0; k < 32; ++k) {  // lanes below 32 take v[k], the others v[k + 32]
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[k]), __float_as_uint(v[k + 32]), false, false);
    v[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) {  // rows of 16 lanes
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[k]), __float_as_uint(v[k + 16]), false, false);
    v[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  auto halve = [&](auto half, auto ctrl) {
    constexpr int kHalf = decltype(half)::value;
    const bool up = lane & kHalf;
#pragma unroll
    for (int k = 0; k < kHalf; ++k) {
      const float keep = up ? v[k + kHalf] : v[k], give = up ? v[k] : v[k + kHalf];
      v[k] = keep + dpp<decltype(ctrl)::value>(give);
    }
  };
  halve(std::integral_constant<int, 8>{}, std::integral_constant<int, 0x128>{});  // row_ror:8
  halve(std::integral_constant<int, 4>{}, std::integral_constant<int, 0x141>{});  // row_half_mirror
  halve(std::integral_constant<int, 2>{}, std::integral_constant<int, 0x4E>{});   // quad_perm 2,3,0,1
  halve(std::integral_constant<int, 1>{}, std::integral_constant<int, 0xB1>{});   // quad_perm 1,0,3,2
  return v[0];
}

// The gradient that each chunk's own outputs send in front of it (P.gends):
// g <- (g + ds C) a from its last token to its first.
template <typename T, int W>
__global__ __launch_bounds__(W * 64) void grad_ends_kernel(const SelectiveRequest P) {
  constexpr int kSlots = kTile * kLanes / 4;
  constexpr int kPer = kSlots > W * 64 ? kSlots / (W * 64) : 1;
  constexpr int kN = W * kNS;
  __shared__ __align__(16) float2 s_step[kTile][kLanes];  // dt, ds
  __shared__ float s_c[kTile][kN];
  const Place p = place_of(P);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t length = length_of(P, p.b);
  const int64_t first = int64_t(p.chunk) * P.chunk_len;
  const int64_t stop = first + P.chunk_len < P.T ? first + P.chunk_len : P.T;
  const int64_t end = length < stop ? length : stop;
  const T* delta = static_cast<const T*>(P.delta);
  const T* z = static_cast<const T*>(P.z);
  const T* dy = static_cast<const T*>(P.dy);
  const T* Cm = static_cast<const T*>(P.Cm);
  const int64_t d = p.c0 + lane;
  const int n0 = wave * kNS;
  const bool mine = lane < p.width;
  float a2[kNS], g[kNS];
#pragma unroll
  for (int i = 0; i < kNS; ++i) {
    a2[i] = mine && n0 + i < P.N ? P.A[d * P.N + n0 + i] * kLog2e : 0.0f;
    g[i] = 0.0f;
  }
  const int64_t tiles = end > first ? (end - first + kTile - 1) / kTile : 0;
  for (int64_t k = tiles - 1; k >= 0; --k) {
    const int64_t t0 = first + k * kTile;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int slot = tid + j * W * 64, at = slot / (kLanes / 4), c4 = slot % (kLanes / 4) * 4;
      const int n = p.width - c4;
      if (slot >= kSlots || n <= 0) continue;
      f32x4 dt{}, ds{};
      if (t0 + at < end) {
        const int64_t row = p.b * P.T + t0 + at, c = p.c0 + c4;
        dt = load4(delta + row * P.ld_delta + c, n);
        if (P.bias) dt += load4(P.bias + c, n);
        ds = load4(dy + row * P.ld_dy + c, n);
        f32x4 zz{};
        if (z) zz = load4(z + row * P.ld_z + c, n);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (P.softplus) dt[e] = softplus_f(dt[e]);
          if (z) ds[e] *= zz[e] * logistic_f(zz[e]);
        }
      }
      f32x4* to = reinterpret_cast<f32x4*>(&s_step[at][c4]);
      to[0] = f32x4{dt[0], ds[0], dt[1], ds[1]};
      to[1] = f32x4{dt[2], ds[2], dt[3], ds[3]};
    }
    for (int i = tid; i < kTile * kN; i += W * 64) {
      const int t = i / kN, n = i % kN;
      s_c[t][n] = t0 + t < end && n < P.N ? to_f32(Cm[(p.b * P.T + t0 + t) * P.ld_c + int64_t(p.group) * P.N + n]) : 0.0f;
    }
    __syncthreads();
    // tokens behind the end have step 0 and gradient 0
#pragma unroll
    for (int t = kTile - 1; t >= 0; --t) {
      const float2 s = s_step[t][lane];
#pragma unroll
      for (int i = 0; i < kNS; ++i) g[i] = fmaf(s.y, s_c[t][n0 + i], g[i]) * __builtin_amdgcn_exp2f(s.x * a2[i]);
    }
  }
  const int64_t m = (int64_t(p.chunk) * P.B + p.b) * P.N;
#pragma unroll
  for (int i = 0; i < kNS; ++i)
    if (mine && n0 + i < P.N) P.gends[(m + n0 + i) * P.D + d] = g[i];
}

// SG: groups of four states that each wave goes through one after another (two
// where N is above 32).
template <typename T, int W, int SG>
__global__ __launch_bounds__(W * 64) void backward_kernel(const SelectiveRequest P) {
  constexpr int kSlots = kTile * kLanes / 4;
  constexpr int kPer = kSlots > W * 64 ? kSlots / (W * 64) : 1;
  constexpr int kN = W * kNS * SG;
  __shared__ __align__(16) f32x4 s_step[kTile][kLanes];  // dt, dt u, ds
  __shared__ float s_b[kTile][kN], s_c[kTile][kN];
  __shared__ __align__(16) float s_write[W][kTile][kLanes];  // the waves' shares of sum G B
  __shared__ __align__(16) float s_decay[W][kTile][kLanes];  // of sum A q
  __shared__ __align__(16) float s_y[W][kTile][kLanes];      // of sum C h
  const Place p = place_of(P);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t length = length_of(P, p.b);
  const int64_t first = int64_t(p.chunk) * P.chunk_len;
  const int64_t stop = first + P.chunk_len < P.T ? first + P.chunk_len : P.T;
  const int64_t end = length < stop ? length : stop;
  const T* u = static_cast<const T*>(P.u);
  const T* delta = static_cast<const T*>(P.delta);
  const T* z = static_cast<const T*>(P.z);
  const T* dy = static_cast<const T*>(P.dy);
  const T* Bm = static_cast<const T*>(P.Bm);
  const T* Cm = static_cast<const T*>(P.Cm);
  T* du = static_cast<T*>(P.du);
  T* ddelta = static_cast<T*>(P.ddelta);
  T* dz = static_cast<T*>(P.dz);
  const int64_t d = p.c0 + lane;
  const bool mine = lane < p.width;
  float a[SG][kNS], G[SG][kNS], start[SG][kNS], dA[SG][kNS];
#pragma unroll
  for (int g = 0; g < SG; ++g)
#pragma unroll
    for (int i = 0; i < kNS; ++i) {
      const int n = (g * W + wave) * kNS + i;
      const bool is = mine && n < P.N;
      const int64_t m = ((int64_t(p.chunk) * P.B + p.b) * P.N + n) * P.D + d, own = (p.b * P.D + d) * P.N + n;
      a[g][i] = is ? P.A[d * P.N + n] : 0.0f;
      start[g][i] = G[g][i] = dA[g][i] = 0.0f;
      if (is && P.chunks > 1) {
        start[g][i] = P.ends[m];
        G[g][i] = P.gends[m];
      } else if (is) {
        if (P.h0) start[g][i] = P.h0[own];
        if (P.dh_last) G[g][i] = P.dh_last[own];
      }
    }
  int at[kPer], c4[kPer];
  f32x4 bias[kPer], skip[kPer], dskip[kPer], dbias[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int slot = tid + j * W * 64;
    at[j] = slot / (kLanes / 4);
    c4[j] = slot % (kLanes / 4) * 4;
    if (slot < kSlots && c4[j] >= p.width) {  // lanes without a channel add zeros to the sums over channels
#pragma unroll
      for (int e = 0; e < 4; ++e) s_step[at[j]][c4[j] + e] = f32x4{};
    }
    if (slot >= kSlots || c4[j] >= p.width) at[j] = kTile;
    bias[j] = skip[j] = dskip[j] = dbias[j] = f32x4{};
    if (at[j] < kTile) {
      if (P.bias) bias[j] = load4(P.bias + p.c0 + c4[j], p.width - c4[j]);
      if (P.skip) skip[j] = load4(P.skip + p.c0 + c4[j], p.width - c4[j]);
    }
  }
  const int64_t parts_row = (int64_t(p.group) * P.tiles_per_group + p.tile) * P.B + p.b;
  const int64_t tiles = end > first ? (end - first + kTile - 1) / kTile : 0;
  f32x4 ru[kPer], rd[kPer], rg[kPer], rz[kPer];
  auto fetch = [&](int64_t t0) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      ru[j] = rd[j] = rg[j] = rz[j] = f32x4{};
      if (at[j] < kTile && t0 + at[j] < end) {
        const int64_t row = p.b * P.T + t0 + at[j], c = p.c0 + c4[j];
        const int n = p.width - c4[j];
        ru[j] = load4(u + row * P.ld_u + c, n);
        rd[j] = load4(delta + row * P.ld_delta + c, n);
        rg[j] = load4(dy + row * P.ld_dy + c, n);
        if (z) rz[j] = load4(z + row * P.ld_z + c, n);
      }
    }
  };
  if (tiles > 0) fetch(first + (tiles - 1) * kTile);
  for (int64_t k = tiles - 1; k >= 0; --k) {
    const int64_t t0 = first + k * kTile;
    const int count = int(end - t0 < kTile ? end - t0 : kTile);
    f32x4 cu[kPer], cx[kPer], cg[kPer], cz[kPer], cdt[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      cu[j] = ru[j];
      cg[j] = rg[j];
      cz[j] = rz[j];
      cx[j] = rd[j] + bias[j];
      if (at[j] >= kTile) continue;
      f32x4 dt = cx[j], ds = cg[j];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (P.softplus) dt[e] = softplus_f(dt[e]);
        if (z) ds[e] *= cz[j][e] * logistic_f(cz[j][e]);
      }
      if (at[j] >= count) dt = f32x4{};  // and u = dy = 0: the state and its gradient pass
      cdt[j] = dt;
#pragma unroll
      for (int e = 0; e < 4; ++e) s_step[at[j]][c4[j] + e] = f32x4{dt[e], dt[e] * cu[j][e], ds[e], 0.0f};
    }
    for (int i = tid; i < kTile * kN; i += W * 64) {
      const int t = i / kN, n = i % kN;
      const bool is = t < count && n < P.N;
      const int64_t row = p.b * P.T + t0 + t, off = int64_t(p.group) * P.N + n;
      s_b[t][n] = is ? to_f32(Bm[row * P.ld_b + off]) : 0.0f;
      s_c[t][n] = is ? to_f32(Cm[row * P.ld_c + off]) : 0.0f;
    }
    if (k > 0) fetch(t0 - kTile);
    __syncthreads();
    const int64_t m = (t0 / kTile * P.B + p.b) * (P.N + 1);
    const float so_far = mine ? P.marks[(m + P.N) * P.D + d] : 0.0f;
#pragma unroll
    for (int g = 0; g < SG; ++g) {
      const int n0 = (g * W + wave) * kNS;
      float h[kNS], hp[kTile][kNS], decay[kTile][kNS], v[64];
#pragma unroll
      for (int i = 0; i < kNS; ++i) {
        h[i] = mine && n0 + i < P.N ? P.marks[(m + n0 + i) * P.D + d] : 0.0f;
        if (start[g][i] != 0.0f)  // a zero state stays zero however its factor overflows
          h[i] = fmaf(__builtin_amdgcn_exp2f(so_far * (a[g][i] * kLog2e)), start[g][i], h[i]);
      }
#pragma unroll
      for (int t = 0; t < kTile; ++t) {
        const f32x4 s = s_step[t][lane];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kNS; ++i) {
          hp[t][i] = h[i];
          decay[t][i] = __builtin_amdgcn_exp2f(s[0] * (a[g][i] * kLog2e));
          h[i] = fmaf(decay[t][i], h[i], s[1] * s_b[t][n0 + i]);
          sum = fmaf(h[i], s_c[t][n0 + i], sum);
          v[t * kNS + i] = s[2] * h[i];
        }
        if (z) s_y[wave][t][lane] = g == 0 ? sum : s_y[wave][t][lane] + sum;
      }
      const int64_t to = ((parts_row * P.T + t0 + lane / kNS) * 2) * kN + n0 + lane % kNS;
      const float dC = sum64(v, lane);
      if (lane / kNS < count) P.parts[to + kN] = dC;
#pragma unroll
      for (int t = kTile - 1; t >= 0; --t) {
        const f32x4 s = s_step[t][lane];
        float through = 0.0f, rate = 0.0f;
#pragma unroll
        for (int i = 0; i < kNS; ++i) {
          G[g][i] = fmaf(s[2], s_c[t][n0 + i], G[g][i]);
          through = fmaf(G[g][i], s_b[t][n0 + i], through);
          v[t * kNS + i] = G[g][i] * s[1];
          G[g][i] *= decay[t][i];
          const float q = G[g][i] * hp[t][i];
          rate = fmaf(q, a[g][i], rate);
          dA[g][i] = fmaf(q, s[0], dA[g][i]);
        }
        s_write[wave][t][lane] = g == 0 ? through : s_write[wave][t][lane] + through;
        s_decay[wave][t][lane] = g == 0 ? rate : s_decay[wave][t][lane] + rate;
      }
      const float dB = sum64(v, lane);
      if (lane / kNS < count) P.parts[to] = dB;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (at[j] >= count) continue;
      f32x4 through{}, rate{}, sum = skip[j] * cu[j], gx, gz;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        through += *reinterpret_cast<const f32x4*>(&s_write[w][at[j]][c4[j]]);
        rate += *reinterpret_cast<const f32x4*>(&s_decay[w][at[j]][c4[j]]);
        if (z) sum += *reinterpret_cast<const f32x4*>(&s_y[w][at[j]][c4[j]]);
      }
      f32x4 ds = cg[j];
      gx = cu[j] * through + rate;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (P.softplus) gx[e] *= logistic_f(cx[j][e]);
        if (z) {
          const float s = logistic_f(cz[j][e]);
          gz[e] = cg[j][e] * sum[e] * (s * fmaf(cz[j][e], 1.0f - s, 1.0f));
          ds[e] *= cz[j][e] * s;
        }
      }
      dskip[j] += ds * cu[j];
      dbias[j] += gx;
      const int64_t o = (p.b * P.T + t0 + at[j]) * P.D + p.c0 + c4[j];
      const int n = p.width - c4[j];
      store4(du + o, cdt[j] * through + skip[j] * ds, n);
      store4(ddelta + o, gx, n);
      if (z) store4(dz + o, gz, n);
    }
  }
  // Rows behind the sequence's end are zero.
  for (int64_t t0 = first > end ? first : end; t0 < stop; t0 += kTile) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (at[j] >= kTile || t0 + at[j] >= stop) continue;
      const int64_t o = (p.b * P.T + t0 + at[j]) * P.D + p.c0 + c4[j];
      const int n = p.width - c4[j];
      store4(du + o, f32x4{}, n);
      store4(ddelta + o, f32x4{}, n);
      if (z) store4(dz + o, f32x4{}, n);
    }
  }
  const int64_t own = p.b * P.chunks + p.chunk;
#pragma unroll
  for (int g = 0; g < SG; ++g)
#pragma unroll
    for (int i = 0; i < kNS; ++i) {
      const int n = (g * W + wave) * kNS + i;
      if (!mine || n >= P.N) continue;
      P.aparts[(own * (P.N + 2) + n) * P.D + d] = dA[g][i];
      if (P.dh0 != nullptr && p.chunk == 0) P.dh0[(p.b * P.D + d) * P.N + n] = G[g][i];
    }
  // The slots' sums over tokens, then over the 16 tokens of a tile.
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (at[j] < kTile) {
      *reinterpret_cast<f32x4*>(&s_write[0][at[j]][c4[j]]) = dskip[j];
      *reinterpret_cast<f32x4*>(&s_decay[0][at[j]][c4[j]]) = dbias[j];
    }
  __syncthreads();
  if (wave == 0 && mine) {
    float sk = 0.0f, bi = 0.0f;
#pragma unroll
    for (int t = 0; t < kTile; ++t) {
      sk += s_write[0][t][lane];
      bi += s_decay[0][t][lane];
    }
    P.aparts[(own * (P.N + 2) + P.N) * P.D + d] = sk;
    P.aparts[(own * (P.N + 2) + P.N + 1) * P.D + d] = bi;
  }
}

// dB and dC from the parts of each 64 channels; `padded` states per row.
template <typename T>
__global__ __launch_bounds__(256) void reduce_tokens_kernel(const SelectiveRequest P, int padded) {
  const int64_t per = int64_t(2) * padded;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;  // [G][B][T][2][padded]
  const int64_t rows = P.B * P.T;
  if (i >= rows * P.G * per) return;
  const int64_t r = i / per % rows, g = i / (per * rows);
  const int w = int(i % per / padded), n = int(i % padded);
  if (n >= P.N) return;
  const bool seen = r % P.T < length_of(P, r / P.T);
  float sum = 0.0f;
  if (seen) {
    const float* src = P.parts + (g * P.tiles_per_group * rows + r) * per + w * padded + n;
    for (int k = 0; k < P.tiles_per_group; ++k) sum += src[k * rows * per];
  }
  T* out = static_cast<T*>(w ? P.dC : P.dB);
  out[(r * P.G + g) * P.N + n] = from_f32<T>(sum);
}

// dA, dskip and dbias from the parts of each sequence and chunk.
__global__ __launch_bounds__(1024) void reduce_channels_kernel(const SelectiveRequest P) {
  column_sums(P.aparts, P.B * P.chunks, int64_t(P.N + 2) * P.D, [&](int64_t c, float sum) {
    const int64_t n = c / P.D, d = c % P.D;  // [N + 2][D]
    if (n < P.N)
      P.dA[d * P.N + n] = sum;
    else if (n == P.N && P.dskip)
      P.dskip[d] = sum;
    else if (n == P.N + 1 && P.dbias)
      P.dbias[d] = sum;
  });
}

template <typename T, int W, int SG>
void launch_main(const SelectiveRequest& P, uint32_t blocks) {
  hipLaunchKernelGGL((backward_kernel<T, W, SG>), dim3(blocks), dim3(W * 64), 0, P.stream, P);
}
template <typename T>
void launch_all(const SelectiveRequest& P) {
  const uint32_t blocks = uint32_t(P.B * P.G * P.tiles_per_group * P.chunks);
  if (P.N <= 4)
    launch_main<T, 1, 1>(P, blocks);
  else if (P.N <= 8)
    launch_main<T, 2, 1>(P, blocks);
  else if (P.N <= 16)
    launch_main<T, 4, 1>(P, blocks);
  else if (P.N <= 32)
    launch_main<T, 8, 1>(P, blocks);
  else
    launch_main<T, 8, 2>(P, blocks);
  const int padded = int(selective_padded(P.N));
  const int64_t n = P.B * P.T * P.G * 2 * padded;
  if (n > 0) hipLaunchKernelGGL(reduce_tokens_kernel<T>, dim3(uint32_t((n + 255) / 256)), dim3(256), 0, P.stream, P, padded);
}
template <typename T>
void launch_ends(const SelectiveRequest& P) {
  const uint32_t blocks = uint32_t(P.B * P.G * P.tiles_per_group * P.chunks);
  auto run = [&](auto* kernel, int W) { hipLaunchKernelGGL(kernel, dim3(blocks), dim3(W * 64), 0, P.stream, P); };
  if (P.N <= 4)
    run(grad_ends_kernel<T, 1>, 1);
  else if (P.N <= 8)
    run(grad_ends_kernel<T, 2>, 2);
  else if (P.N <= 16)
    run(grad_ends_kernel<T, 4>, 4);
  else if (P.N <= 32)
    run(grad_ends_kernel<T, 8>, 8);
  else
    run(grad_ends_kernel<T, 16>, 16);
}

sr_status launched(const char* what) {
  const hipError_t err = hipGetLastError();
  return err == hipSuccess ? SR_OK : fail(SR_ERR_HIP, "%s: %s", what, hipGetErrorString(err));
}

}  // namespace

sr_status launch_selective_backward(const SelectiveRequest& P) {
  sr_status st = P.B > 0 ? launch_selective_states(P) : SR_OK;
  if (st != SR_OK) return st;
  if (P.B > 0 && P.chunks > 1) {
    st = launch_selective_carry(P, P.h0, nullptr, false);
    if (st != SR_OK) return st;
    if (P.dtype == SR_BF16)
      launch_ends<uint16_t>(P);
    else
      launch_ends<float>(P);
    st = launched("selective scan gradients");
    if (st != SR_OK) return st;
    SelectiveRequest back = P;
    back.ends = P.gends;
    st = launch_selective_carry(back, P.dh_last, nullptr, true);
    if (st != SR_OK) return st;
  }
  if (P.B > 0) {
    if (P.dtype == SR_BF16)
      launch_all<uint16_t>(P);
    else
      launch_all<float>(P);
    st = launched("selective scan backward");
    if (st != SR_OK) return st;
  }
  const int64_t n = int64_t(P.N + 2) * P.D;
  hipLaunchKernelGGL(reduce_channels_kernel, dim3(uint32_t((n + 63) / 64)), dim3(1024), 0, P.stream, P);
  return launched("selective scan gradient sums");
}

}  // namespace sr
