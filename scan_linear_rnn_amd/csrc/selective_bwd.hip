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
// The states are computed again from marks: the forward's first pass (scan_kernel
// with kMarks) writes what each chunk has made of a zero state in front of
// every 16 tokens, and the sum of its steps there, so that the state itself is one
// exponential and one product away from the chunk's start.  A workgroup then owns
// 64 channels of one chunk, a lane each, goes back over its tiles of 16
// tokens, runs each forward into registers and back again; its eight waves hold two
// states per lane each (four of one or two up to eight states; above 16 each wave goes through
// two or four such groups of states, whose forward walk is repeated for each half of
// a tile).  The sums over channels, dB and dC, are 32 values each per wave and half
// tile (8 tokens, 2 states, both) to be summed over 64 lanes: a halving exchange (swaps of
// half waves, then of rows, then DPP) leaves one sum in every lane at about two
// instructions per value, where separate sums would take six.  They go out per 64
// channels and reduce_tokens_kernel adds those up, always in the same order.
//
// 8 x 2048 x 1024, 16 states, gated, bf16: 456 us, of them marks 65, the gradients in front of
// the chunks 63, two carries 10, this kernel 340 to 354 (traced), sums 16.  Its vector units are busy
// for 65% of its time: 123 KB of LDS per workgroup and 232 registers per lane, each of which by itself leaves a
// SIMD two waves to choose from.  32 states 1.0 ms (27 registers spilled); 64 states, whose groups do not fit the
// registers (165 to 196 spilled), 3.1 ms.

#include "layer_util.hpp"

namespace sr {
namespace {

template <int kCtrl>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(
      uint32_t(__builtin_amdgcn_mov_dpp(int(__float_as_uint(x)), kCtrl, 0xF, 0xF, true)));
}

// One stage of sum_lanes: every lane adds the partner's number at lane ^ kBit (or, for 4,
// at the mirrored place of its eight lanes), and of two numbers keeps one half of the sums.
template <int kBit, int n>
__device__ __forceinline__ void sum_stage(float (&v)[n], int lane) {
  constexpr int kLeft = n > 64 ? 0 : n;
  constexpr int kHalf = kLeft * kBit / 64;  // numbers left after this stage, none: one in several lanes
  auto partner = [](float x) {
    if constexpr (kBit == 8) return dpp<0x128>(x);  // row_ror:8
    if constexpr (kBit == 4) return dpp<0x141>(x);  // row_half_mirror
    if constexpr (kBit == 2) return dpp<0x4E>(x);   // quad_perm 2,3,0,1
    return dpp<0xB1>(x);                            // quad_perm 1,0,3,2
  };
  if constexpr (kHalf == 0) {
    v[0] += partner(v[0]);
  } else {
#pragma unroll
    for (int k = 0; k < kHalf; ++k) {
      if constexpr (kBit == 32) {  // lanes below 32 keep v[k], the others v[k + kHalf]
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[k]), __float_as_uint(v[k + kHalf]), false, false);
        v[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
      } else if constexpr (kBit == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[k]), __float_as_uint(v[k + kHalf]), false, false);
        v[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
      } else {
        const bool up = lane & kBit;
        const float keep = up ? v[k + kHalf] : v[k], give = up ? v[k] : v[k + kHalf];
        v[k] = keep + partner(give);
      }
    }
  }
}
// Sums of n values (8, 16 or 32) over the 64 lanes: lane l returns the sum of v[l n / 64].
template <int n>
__device__ __forceinline__ float sum_lanes(float (&v)[n], int lane) {
  sum_stage<32>(v, lane);
  sum_stage<16>(v, lane);
  sum_stage<8>(v, lane);
  sum_stage<4>(v, lane);
  sum_stage<2>(v, lane);
  sum_stage<1>(v, lane);
  return v[0];
}

// The gradient that each chunk's own outputs send in front of it (P.gends):
// g <- (g + ds C) a from its last token to its first.  Tiles as in scan_kernel, last one first.
template <typename T, int W, int NS, bool kWhole>
__global__ __launch_bounds__(W * 64) void grad_ends_kernel(const SelectiveRequest P) {
  constexpr int Q = kTile / W;
  __shared__ __align__(16) float2 s_step[2][kTile][kLanes];  // dt, ds
  const Place p = place_of(P);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t length = length_of(P, p.b);
  const int64_t first = int64_t(p.chunk) * P.chunk_len;
  const int64_t stop = first + P.chunk_len < P.T ? first + P.chunk_len : P.T;
  const int64_t end = length < stop ? length : stop;
  const int64_t d = p.c0 + lane;
  const int n0 = wave * NS;
  const bool mine = lane < p.width;
  float a2[NS], g[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    a2[i] = mine && n0 + i < P.N ? rate2(P.A[d * P.N + n0 + i]) : 0.0f;
    g[i] = 0.0f;
  }
  const int at = tid / (kLanes / Q), lc = tid % (kLanes / Q) * Q;
  const int c = lc < p.width ? lc : 0, nc = p.width - c, bc_at = lane % 16;
  const int64_t group0 = int64_t(p.group) * P.N + (n0 < P.N ? n0 : 0);
  const int nn = n0 < P.N ? P.N - n0 : 1;
  float bias[Q];
  load_some(P.bias + p.c0 + c, P.bias ? nc : 0, bias);
  struct Inputs {
    Raw<T, Q> delta, dy, z;
    Raw<T, NS> Cm;
  };
  auto fetch = [&](int64_t t0, Inputs& in) {
    t0 = t0 < first ? first : t0;
    const int64_t row0 = p.b * P.T + t0;
    const int last = int(P.T - 1 - t0), t = at < last ? at : last, tb = bc_at < last ? bc_at : last;
    load_raw<kWhole>(at_byte(static_cast<const T*>(P.delta) + row0 * P.ld_delta + p.c0, row_bytes<T>(t, P.ld_delta, c)), nc, in.delta);
    load_raw<kWhole>(at_byte(static_cast<const T*>(P.dy) + row0 * P.ld_dy + p.c0, row_bytes<T>(t, P.ld_dy, c)), nc, in.dy);
    if (P.z) load_raw<kWhole>(at_byte(static_cast<const T*>(P.z) + row0 * P.ld_z + p.c0, row_bytes<T>(t, P.ld_z, c)), nc, in.z);
    load_raw<kWhole>(at_byte(static_cast<const T*>(P.Cm) + row0 * P.ld_c + group0, row_bytes<T>(tb, P.ld_c, 0)), nn, in.Cm);
  };
  auto prepare = [&](int64_t t0, int buffer, const Inputs& in, float (&cm)[NS]) {
    float dt[Q], ds[Q], z[Q];
    values(in.delta, dt);
    values(in.dy, ds);
#pragma unroll
    for (int e = 0; e < Q; ++e) dt[e] += bias[e];
    if (P.softplus) {
#pragma unroll
      for (int e = 0; e < Q; ++e) dt[e] = softplus_f(dt[e]);
    }
    if (P.z) {
      values(in.z, z);
#pragma unroll
      for (int e = 0; e < Q; ++e) ds[e] *= z[e] * logistic_f(z[e]);
    }
    values(in.Cm, cm);
    if (t0 + kTile > end) {  // tokens behind the end have step 0 and gradient 0
#pragma unroll
      for (int e = 0; e < Q; ++e)
        if (t0 + at >= end) dt[e] = ds[e] = 0.0f;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (t0 + bc_at >= end) cm[i] = 0.0f;
    }
    if (!kWhole || n0 >= P.N) {
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (n0 + i >= P.N) cm[i] = 0.0f;
    }
    float pair[2 * Q];
#pragma unroll
    for (int e = 0; e < Q; ++e) {
      pair[2 * e] = dt[e];
      pair[2 * e + 1] = ds[e];
    }
    __builtin_memcpy(__builtin_assume_aligned(&s_step[buffer][at][lc], Q > 1 ? 16 : 8), pair, 8 * Q);
  };
  Inputs in[2];
  float c0[NS];
  auto tile = [&](auto parity, int64_t t0) {
    constexpr int s = decltype(parity)::value;
    float2 step[kTile];
#pragma unroll
    for (int t = 0; t < kTile; ++t) step[t] = s_step[s][t][lane];
    float cm[NS];
    prepare(t0 - kTile, s ^ 1, in[s], cm);
    fetch(t0 - 3 * kTile, in[s]);
    unrolled<kTile>([&](auto token) {
      constexpr int t = kTile - 1 - decltype(token)::value;
      row_add<t>(c0, step[t].y, g);
#pragma unroll
      for (int i = 0; i < NS; ++i) g[i] *= __builtin_amdgcn_exp2f(step[t].x * a2[i]);
    });
#pragma unroll
    for (int i = 0; i < NS; ++i) c0[i] = cm[i];
    __syncthreads();
  };
  if (first < end) {
    int64_t t0 = first + (end - 1 - first) / kTile * kTile;
    fetch(t0, in[1]);
    fetch(t0 - kTile, in[0]);
    prepare(t0, 0, in[1], c0);
    fetch(t0 - 2 * kTile, in[1]);
    __syncthreads();
    for (; t0 - kTile >= first; t0 -= 2 * kTile) {
      tile(std::integral_constant<int, 0>{}, t0);
      tile(std::integral_constant<int, 1>{}, t0 - kTile);
    }
    if (t0 >= first) tile(std::integral_constant<int, 0>{}, t0);
  }
  const int64_t m = (int64_t(p.chunk) * P.B + p.b) * P.N;
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (mine && n0 + i < P.N) P.gends[(m + n0 + i) * P.D + d] = g[i];
}

// W waves of NS states per lane; SG: groups of W NS states that the waves go
// through one after another.  Each wave prepares and finishes the tokens wave, wave + W,
// .. of a tile, a channel per lane.  A tile takes two phases with a barrier each: its
// states forwards and the gradients of its later eight tokens, then those of the
// earlier eight; the next tile's steps are prepared, and the outputs of the eight
// tokens before are finished, in between.
template <typename T, int W, int NS, int SG, bool kGated>
__global__ __launch_bounds__(W * 64, 2) void backward_kernel(const SelectiveRequest P) {
  constexpr int kN = W * NS * SG, kV = 8 * NS, kOwn = kTile / W, kHalf = kOwn / 2;
  __shared__ float2 s_step[2][kTile][kLanes];                  // dt, dt u
  __shared__ float s_ds[2][kTile][kLanes];
  __shared__ float s_write[2][W][8][kLanes];                   // the waves' shares of sum G B
  __shared__ float s_decay[2][W][8][kLanes];                   // of sum A q
  __shared__ float s_y[2][W][8][kLanes];                       // of sum C h
  const Place p = place_of(P);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t length = length_of(P, p.b);
  const int64_t first = int64_t(p.chunk) * P.chunk_len;
  const int64_t stop = first + P.chunk_len < P.T ? first + P.chunk_len : P.T;
  const int64_t end = length < stop ? length : stop;
  const bool mine = lane < p.width;
  const int c = mine ? lane : 0, bc_at = lane % 16;
  const int64_t d = p.c0 + c;
  float a[SG][NS], G[SG][NS], start[SG][NS], dA[SG][NS];
#pragma unroll
  for (int g = 0; g < SG; ++g)
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int n = (g * W + wave) * NS + i;
      const bool is = mine && n < P.N;
      const int64_t m = ((int64_t(p.chunk) * P.B + p.b) * P.N + n) * P.D + d, own = (p.b * P.D + d) * P.N + n;
      a[g][i] = is ? bounded(P.A[d * P.N + n]) : 0.0f;
      start[g][i] = G[g][i] = dA[g][i] = 0.0f;
      if (is && P.chunks > 1) {
        start[g][i] = P.ends[m];
        G[g][i] = P.gends[m];
      } else if (is) {
        if (P.h0) start[g][i] = P.h0[own];
        if (P.dh_last) G[g][i] = P.dh_last[own];
      }
    }
  const float bias = P.bias ? P.bias[d] : 0.0f, skip = P.skip ? P.skip[d] : 0.0f;
  float dskip = 0.0f, dbias = 0.0f;
  // A tile's inputs as they stand in memory, and the states in front of it.
  struct Inputs {
    T u[kOwn], delta[kOwn], dy[kOwn], z[kOwn];
    T Bm[SG][NS], Cm[SG][NS];
    float mark[SG][NS], so_far;
  } in;
  auto fetch = [&](int64_t t0) {
    t0 = t0 > first ? t0 : first;
    const int64_t row0 = p.b * P.T + t0;
    const int last = int(P.T - 1 - t0), tb = bc_at < last ? bc_at : last;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const int t = wave + j * W < last ? wave + j * W : last;  // (uniform)
      in.u[j] = (static_cast<const T*>(P.u) + (row0 + t) * P.ld_u + p.c0)[c];
      in.delta[j] = (static_cast<const T*>(P.delta) + (row0 + t) * P.ld_delta + p.c0)[c];
      in.dy[j] = (static_cast<const T*>(P.dy) + (row0 + t) * P.ld_dy + p.c0)[c];
      if (kGated) in.z[j] = (static_cast<const T*>(P.z) + (row0 + t) * P.ld_z + p.c0)[c];
    }
    const int64_t m = (t0 / kTile * P.B + p.b) * (P.N + 1);
    in.so_far = (P.marks + (m + P.N) * P.D + p.c0)[c];
#pragma unroll
    for (int g = 0; g < SG; ++g) {
      const int n0 = (g * W + wave) * NS;
      const T *Bm = static_cast<const T*>(P.Bm) + row0 * P.ld_b + int64_t(p.group) * P.N,
              *Cm = static_cast<const T*>(P.Cm) + row0 * P.ld_c + int64_t(p.group) * P.N;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int n = n0 + i < P.N ? n0 + i : P.N - 1;  // (uniform)
        in.Bm[g][i] = *at_byte(Bm + n, row_bytes<T>(tb, P.ld_b, 0));
        in.Cm[g][i] = *at_byte(Cm + n, row_bytes<T>(tb, P.ld_c, 0));
      }
#pragma unroll
      for (int i = 0; i < NS; ++i) in.mark[g][i] = (P.marks + (m + (n0 + i < P.N ? n0 + i : P.N)) * P.D + p.c0)[c];
    }
  };
  struct Tokens {
    float u[kOwn], x[kOwn], dy[kOwn], z[kOwn], dt[kOwn];
  };
  struct States {
    float b[SG][NS], c[SG][NS], h[SG][NS];
  };
  // Converts what was fetched for the tile at t0 and writes its steps.
  auto prepare = [&](int64_t t0, int buffer, Tokens& k, States& n) {
    const int count = int(end - t0 < kTile ? end - t0 : kTile);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const int t = wave + j * W;
      const bool live = mine && t < count;  // what does not exist adds zeros, and the state passes
      k.u[j] = live ? to_f32(in.u[j]) : 0.0f;
      k.x[j] = to_f32(in.delta[j]) + bias;
      k.dy[j] = live ? to_f32(in.dy[j]) : 0.0f;
      const float soft = softplus_f(k.x[j]);
      k.dt[j] = !mine || t >= count ? 0.0f : P.softplus ? soft : k.x[j];
      float ds = k.dy[j];
      if (kGated) {
        k.z[j] = live ? to_f32(in.z[j]) : 0.0f;
        ds *= k.z[j] * logistic_f(k.z[j]);
      }
      s_step[buffer][t][lane] = float2{k.dt[j], k.dt[j] * k.u[j]};
      s_ds[buffer][t][lane] = ds;
    }
#pragma unroll
    for (int g = 0; g < SG; ++g) {
      const int n0 = (g * W + wave) * NS;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const bool is = bc_at < count && n0 + i < P.N;
        n.b[g][i] = is ? to_f32(in.Bm[g][i]) : 0.0f;
        n.c[g][i] = is ? to_f32(in.Cm[g][i]) : 0.0f;
        n.h[g][i] = mine && n0 + i < P.N ? in.mark[g][i] : 0.0f;
        // a zero state stays zero however its factor overflows
        // of several groups the walk's own rates: others in registers beside them spill (64 states 3.26 ms, so 3.11)
        const float half = SG > 1 ? 0.5f * (in.so_far * rate2(a[g][i])) : in.so_far * half_rate2(a[g][i]);
        const float full = decayed(half, start[g][i], n.h[g][i]);
        n.h[g][i] = start[g][i] != 0.0f ? full : n.h[g][i];
      }
    }
  };
  // The waves' shares for a thread's tokens in a half of a tile, read ahead of their use.
  struct Shares {
    float write[kHalf][W], decay[kHalf][W], y[kHalf][kGated ? W : 1];
  };
  auto collect = [&](auto half, Shares& s) {
    constexpr int kSide = decltype(half)::value;
#pragma unroll
    for (int j = 0; j < kHalf; ++j)
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const int r = wave + j * W;
        s.write[j][w] = s_write[kSide][w][r][lane];
        s.decay[j][w] = s_decay[kSide][w][r][lane];
        if (kGated) s.y[j][w] = s_y[kSide][w][r][lane];
      }
    __builtin_amdgcn_sched_barrier(0);  // where they stand: a wait for each would follow else
  };
  // The gradients of a thread's tokens in the half of the tile at t0.
  auto finish = [&](int64_t t0, auto half, const Tokens& k, const Shares& shares) {
    constexpr int kSide = decltype(half)::value;
#pragma unroll
    for (int jj = 0; jj < kHalf; ++jj) {
      const int j = kSide * kHalf + jj, t = wave + j * W;
      float through = 0.0f, rate = 0.0f, sum = skip * k.u[j];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        through += shares.write[jj][w];
        rate += shares.decay[jj][w];
        if (kGated) sum += shares.y[jj][w];
      }
      float ds = k.dy[j], gz = 0.0f, gx = fmaf(k.u[j], through, rate);
      if (kGated) {
        const float s = logistic_f(k.z[j]);
        gz = k.dy[j] * sum * (s * fmaf(k.z[j], 1.0f - s, 1.0f));
        ds *= k.z[j] * s;
      }
      const float slope = logistic_f(k.x[j]);
      gx *= P.softplus ? slope : 1.0f;
      const bool live = t0 + t < end && mine;
      const int64_t row = (p.b * P.T + t0 + t) * P.D + p.c0;
      const uint32_t at = live ? uint32_t(lane) * uint32_t(sizeof(T)) : kNowhere;
      const float gu[1] = {fmaf(k.dt[j], through, skip * ds)}, gd[1] = {gx}, gate[1] = {gz};
      store_at(static_cast<T*>(P.du) + row, at, gu);
      store_at(static_cast<T*>(P.ddelta) + row, at, gd);
      if (kGated) store_at(static_cast<T*>(P.dz) + row, at, gate);
      dskip = live ? fmaf(ds, k.u[j], dskip) : dskip;
      dbias = live ? dbias + gx : dbias;
    }
  };
  const int64_t parts_row = (int64_t(p.group) * P.tiles_per_group + p.tile) * P.B + p.b;
  const int64_t last_tile = first + (end - 1 - first) / kTile * kTile;
  constexpr std::integral_constant<int, 0> kEarly{};
  constexpr std::integral_constant<int, 1> kLate{};
  Tokens now, before{};  // of the present tile and the one that came before it, which is later in time
  States n;
  if (first < end) {
    fetch(last_tile);
    prepare(last_tile, 0, now, n);
    fetch(last_tile - kTile);
    __syncthreads();
  }
  int buffer = 0;
  for (int64_t t0 = last_tile; first < end && t0 >= first; t0 -= kTile, buffer ^= 1) {
    const int count = int(end - t0 < kTile ? end - t0 : kTile);
    float2 step[kTile];
    float ds_of[kTile];
#pragma unroll
    for (int t = 0; t < kTile; ++t) {
      step[t] = s_step[buffer][t][lane];
      ds_of[t] = s_ds[buffer][t][lane];
    }
    // The states of group g before and behind the tile's tokens, and their factors.
    struct Walk {
      float h[kTile + 1][NS], decay[kTile][NS];
    } walk;
    auto forward = [&](int g, auto tokens, Walk& w) {
      float a2[NS];
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        w.h[0][i] = n.h[g][i];
        a2[i] = rate2(a[g][i]);
        if constexpr (SG > 1) asm volatile("" : "+v"(a2[i]));  // computed again, not kept
      }
      unrolled<decltype(tokens)::value>([&](auto token) {
        constexpr int t = decltype(token)::value;
        const float2 s = step[t];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          w.decay[t][i] = __builtin_amdgcn_exp2f(s.x * a2[i]);
          w.h[t + 1][i] = fmaf(w.decay[t][i], w.h[t][i], row_times<t>(n.b[g][i], s.y));
        }
      });
    };
    if constexpr (SG == 1) forward(0, std::integral_constant<int, kTile>{}, walk);
    // Back over eight tokens; their products for dB and dC take the registers that
    // their states and decays leave.
    auto back = [&](auto half) {
      constexpr int kSide = decltype(half)::value;
#pragma unroll
      for (int g = 0; g < SG; ++g) {
        if constexpr (SG > 1) {  // the registers hold one group's states at a time
          __builtin_amdgcn_sched_barrier(0);
          forward(g, std::integral_constant<int, kSide ? kTile : kTile / 2>{}, walk);
        }
        float vb[kV], vc[kV];
        unrolled<8>([&](auto token) {
          constexpr int k = 7 - decltype(token)::value, t = 8 * kSide + k;
          const float2 s = step[t];
          const float ds = ds_of[t];
          row_add<t>(n.c[g], ds, G[g]);
          const float through = row_dot<t>(n.b[g], G[g]);
          float rate = 0.0f;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            vc[k * NS + i] = ds * walk.h[t + 1][i];
            vb[k * NS + i] = G[g][i] * s.y;
            G[g][i] *= walk.decay[t][i];
            const float q = G[g][i] * walk.h[t][i];
            rate = fmaf(q, a[g][i], rate);
            dA[g][i] = fmaf(q, s.x, dA[g][i]);
          }
          s_write[kSide][wave][k][lane] = g == 0 ? through : s_write[kSide][wave][k][lane] + through;
          s_decay[kSide][wave][k][lane] = g == 0 ? rate : s_decay[kSide][wave][k][lane] + rate;
          if (kGated) {
            const float sum = row_dot<t>(n.c[g], walk.h[t + 1]);
            s_y[kSide][wave][k][lane] = g == 0 ? sum : s_y[kSide][wave][k][lane] + sum;
          }
        });
        // lane l has the sums of value l kV / 64: of token l kV / 64 / NS, state l kV / 64 % NS
        const float dC = sum_lanes(vc, lane), dB = sum_lanes(vb, lane);
        const int k = lane * kV / 64, t = 8 * kSide + k / NS;
        const uint32_t to = lane % (64 / kV) == 0 && t < count ? uint32_t(t * 2 * kN + k % NS) * 4 : kNowhere;
        float* part = P.parts + ((parts_row * P.T + t0) * 2) * kN + (g * W + wave) * NS;
        const float gb[1] = {dB}, gc[1] = {dC};
        store_at(part, to, gb);
        store_at(part + kN, to, gc);
      }
    };
    Shares shares;
    collect(kEarly, shares);
    back(kLate);
    finish(t0 + kTile, kEarly, before, shares);  // (nothing behind the last tile)
    __syncthreads();
    collect(kLate, shares);
    back(kEarly);
    finish(t0, kLate, now, shares);
    before = now;
    prepare(t0 - kTile, buffer ^ 1, now, n);  // (in front of the first tile: of no use)
    fetch(t0 - 2 * kTile);
    __syncthreads();
  }
  if (first < end) {
    Shares shares;
    collect(kEarly, shares);
    finish(first, kEarly, before, shares);
  }
  // Rows behind the sequence's end are zero.
  for (int64_t t = (first > end ? first : end) + wave; t < stop; t += W) {
    const int64_t row = (p.b * P.T + t) * P.D + p.c0;
    if (!mine) continue;
    (static_cast<T*>(P.du) + row)[c] = T(0);
    (static_cast<T*>(P.ddelta) + row)[c] = T(0);
    if (kGated) (static_cast<T*>(P.dz) + row)[c] = T(0);
  }
  const int64_t own = p.b * P.chunks + p.chunk;
#pragma unroll
  for (int g = 0; g < SG; ++g)
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int k = (g * W + wave) * NS + i;
      if (!mine || k >= P.N) continue;
      P.aparts[(own * (P.N + 2) + k) * P.D + d] = dA[g][i];
      if (P.dh0 != nullptr && p.chunk == 0) P.dh0[(p.b * P.D + d) * P.N + k] = G[g][i];
    }
  // The waves' sums over their tokens.
  __syncthreads();
  s_write[0][wave][0][lane] = dskip;
  s_write[0][wave][1][lane] = dbias;
  __syncthreads();
  if (wave == 0 && mine) {
    float sk = 0.0f, bi = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      sk += s_write[0][w][0][lane];
      bi += s_write[0][w][1][lane];
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
  if (out != nullptr) out[(r * P.G + g) * P.N + n] = from_f32<T>(sum);  // (may be null without channels)
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

sr_status launched(const char* what) {
  const hipError_t err = hipGetLastError();
  return err == hipSuccess ? SR_OK : fail(SR_ERR_HIP, "%s: %s", what, hipGetErrorString(err));
}

template <typename T>
void launch_all(const SelectiveRequest& P) {
  const uint32_t blocks = uint32_t(P.B * P.G * P.tiles_per_group * P.chunks);
  auto either = [&](auto* gated, auto* plain, int w) {
    if (P.z)
      hipLaunchKernelGGL(gated, dim3(blocks), dim3(w * 64), 0, P.stream, P);
    else
      hipLaunchKernelGGL(plain, dim3(blocks), dim3(w * 64), 0, P.stream, P);
  };
  if (P.N <= 4)
    either(backward_kernel<T, 4, 1, 1, true>, backward_kernel<T, 4, 1, 1, false>, 4);
  else if (P.N <= 8)
    either(backward_kernel<T, 4, 2, 1, true>, backward_kernel<T, 4, 2, 1, false>, 4);
  else if (P.N <= 16)
    either(backward_kernel<T, 8, 2, 1, true>, backward_kernel<T, 8, 2, 1, false>, 8);
  else if (P.N <= 32)
    either(backward_kernel<T, 8, 2, 2, true>, backward_kernel<T, 8, 2, 2, false>, 8);
  else
    either(backward_kernel<T, 8, 2, 4, true>, backward_kernel<T, 8, 2, 4, false>, 8);
}
sr_status launch_reduce_tokens(const SelectiveRequest& P) {
  const int padded = int(selective_padded(P.N));
  const int64_t n = P.B * P.T * P.G * 2 * padded;
  if (n == 0) return SR_OK;
  auto run = [&](auto* kernel) {
    hipLaunchKernelGGL(kernel, dim3(uint32_t((n + 255) / 256)), dim3(256), 0, P.stream, P, padded);
  };
  if (P.dtype == SR_BF16)
    run(reduce_tokens_kernel<uint16_t>);
  else
    run(reduce_tokens_kernel<float>);
  return launched("selective scan gradient sums over channels");
}
template <typename T, int W, int NS>
void launch_ends(const SelectiveRequest& P) {
  const uint32_t blocks = uint32_t(P.B * P.G * P.tiles_per_group * P.chunks);
  auto run = [&](auto* kernel) { hipLaunchKernelGGL(kernel, dim3(blocks), dim3(W * 64), 0, P.stream, P); };
  if (P.D / P.G % (kTile / W) == 0 && P.N % NS == 0)
    run(grad_ends_kernel<T, W, NS, true>);
  else
    run(grad_ends_kernel<T, W, NS, false>);
}
template <typename T>
void launch_ends(const SelectiveRequest& P) {
  if (P.N <= 4)
    launch_ends<T, 4, 1>(P);
  else if (P.N <= 8)
    launch_ends<T, 4, 2>(P);
  else if (P.N <= 16)
    launch_ends<T, 4, 4>(P);
  else if (P.N <= 32)
    launch_ends<T, 8, 4>(P);
  else
    launch_ends<T, 8, 8>(P);
}

}  // namespace

sr_status launch_selective_backward(const SelectiveRequest& P) {
  if (P.D == 0) return launch_reduce_tokens(P);  // zeros: sums of no channels
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
    if (st == SR_OK) st = launch_reduce_tokens(P);
    if (st != SR_OK) return st;
  }
  const int64_t n = int64_t(P.N + 2) * P.D;
  hipLaunchKernelGGL(reduce_channels_kernel, dim3(uint32_t((n + 63) / 64)), dim3(1024), 0, P.stream, P);
  return launched("selective scan gradient sums");
}

}  // namespace sr
