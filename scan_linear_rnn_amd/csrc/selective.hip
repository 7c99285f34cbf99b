// The selective state space scan over a sequence, and its single-token step.
//
//     dt = softplus(delta + bias)                      (or delta + bias)
//     h_n <- exp(dt A_n) h_n + (dt u) B_n              n = 1..N, per channel
//     y  = (sum_n C_n h_n + skip u) silu(z)
//
// with A per channel and state, and B, C per token (shared by the channels of
// a group).  States, sums and gates are fp32; y is rounded once.
//
// A workgroup owns 64 channels (a lane each) of one sequence and walks over its
// tokens in tiles of 16; its waves hold one to eight states per lane each (four
// waves of four for 16 states).  B and C go from memory to lanes, token t in lane t of
// each row of 16, and from there into products as operands across lanes.  The
// waves share what is per token and channel: each prepares a part of the
// tile's steps (softplus and the like) in LDS, and sums its part of the waves'
// shares of y.  So every input is read once, wide, and the recurrence, 16 x (2
// products, exp, 2 fused multiply-adds), is what the vector units spend their time on.
//
// Where there are too few sequences and channels to fill the GPU, the tokens are
// cut into chunks: a first pass (kEnds) computes what each chunk adds to a
// zero state and the sum of its steps, whose exponential is the chunk's decay; one
// thread per state then carries the states over the chunks (carry_kernel); and the
// full pass starts each chunk from its own state.
//
// 8 x 4096 x 2048, 16 states, gated, bf16: 351 to 366 us (1.5 TB/s, 3.0e12 states a second).  A
// workgroup per CU, one wave per SIMD: about 455 vector instructions per wave and tile, 64 of
// them exponentials at two slots, which keep its unit active for 67% of the time (a probe of the
// recurrence with the sum over states alone takes 190 us); the rest is waits that no other wave fills.
// Eight waves of two states take as long, 353 us, and more where a CU has several workgroups:
// 16 x 2048 x 2048 292 us with four waves, 358 with eight; 1 x 65536 x 1024 in 96 chunks 465 and 587
// (four waves under a tracer: first pass 212, carry 17, outputs 298, whose vector units are 92% active).

#include "layer_util.hpp"

namespace sr {
namespace {

enum Pass {
  kOutputs,  // y from the chunk's own start state, and the last state
  kEnds,     // the state that the chunk's tokens make of zero, and the sum of their steps
  kMarks,    // and what the chunk has made of zero in front of each tile, with the steps so far
};

// W waves of NS states per lane.
//
// While the waves go through tile k, each thread also prepares its part of tile
// k + 1's steps, sums its part of tile k - 1's outputs and has the inputs of tiles k + 2 and
// k + 3 on their way: everything between two barriers is independent, one barrier per tile.  Tiles with
// four whole ones behind them go without a branch, as one block that the compiler can order.
template <typename T, int W, int NS, int kPass, bool kWhole, bool kGated>
__global__ __launch_bounds__(W * 64, kPass != kOutputs && NS < 8 ? 3 : 2) void scan_kernel(const SelectiveRequest P) {
  constexpr bool kStates = kPass != kOutputs;
  constexpr int Q = kTile / W;  // neighbouring channels of a token that a thread prepares
  __shared__ __align__(16) float2 s_step[2][kTile][kLanes];  // dt, dt u
  __shared__ __align__(16) float s_y[2][kStates ? 1 : W][kTile][kLanes];
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
  // Where N is less than the waves hold, the places behind the last state repeat states and take a
  // part of their C: kWhole, whole waves those of the last wave that has any (an eighth
  // each), else each the last state (a 64th), and what is repeated keeps the rest.  (With zeros for
  // B and C an infinite input would make them NaN, and y with them.)
  const int from = kWhole ? (n0 < P.N ? n0 : P.N - NS) : (n0 < P.N ? n0 : P.N - 1);  // the wave's first state
  const float part_of = kWhole ? 0.125f : 0.015625f;
  const float rest_of = 1.0f - part_of * float(kWhole ? W - P.N / NS : W * NS - P.N);
  const bool shares = P.N < W * NS && n0 + NS >= P.N;
  float a2[NS], h[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = kWhole || from + i < P.N ? from + i : P.N - 1;
    a2[i] = mine ? rate2(P.A[d * P.N + n]) : 0.0f;
    h[i] = 0.0f;
    if constexpr (!kStates) {
      if (P.ends != nullptr) {  // [chunk][b][n][D]
        if (mine) h[i] = P.ends[((int64_t(p.chunk) * P.B + p.b) * P.N + n) * P.D + d];
      } else if (P.h0 != nullptr && mine) {
        h[i] = P.h0[(p.b * P.D + d) * P.N + n];
      }
    }
  }

  const int at = tid / (kLanes / Q), lc = tid % (kLanes / Q) * Q;  // a thread's token in the tile and first lane
  const int c = lc < p.width ? lc : 0;                             // its channel; lanes without one repeat the first
  const int nc = p.width - c;
  float bias[Q], skip[Q];
  load_some(P.bias + p.c0 + c, P.bias ? nc : 0, bias);
  load_some(P.skip + p.c0 + c, !kStates && P.skip ? nc : 0, skip);
  // B and C go from memory to where the recurrence takes them from: lane t of each
  // row of 16 has the wave's states of a tile's token t.
  const int bc_at = lane % 16;
  const int64_t group0 = int64_t(p.group) * P.N + from;
  const int nn = P.N - from;
  struct Inputs {
    Raw<T, Q> u, delta, z;
    Raw<T, NS> Bm, Cm;
  };
  const auto bytes = [](int t, int64_t ld, int i) { return row_bytes<T>(t, ld, i); };
  const uint32_t o_u = bytes(at, P.ld_u, c), o_d = bytes(at, P.ld_delta, c), o_z = bytes(at, P.ld_z, c),
                 o_b = bytes(bc_at, P.ld_b, 0), o_c = bytes(bc_at, P.ld_c, 0);
  const int64_t row0 = p.b * P.T + first;
  const T *pu = static_cast<const T*>(P.u) + row0 * P.ld_u + p.c0, *pd = static_cast<const T*>(P.delta) + row0 * P.ld_delta + p.c0,
          *pz = static_cast<const T*>(P.z) + row0 * P.ld_z + p.c0, *pb = static_cast<const T*>(P.Bm) + row0 * P.ld_b + group0,
          *pc = static_cast<const T*>(P.Cm) + row0 * P.ld_c + group0;  // at `ahead`, the tile that is fetched next
  int64_t ahead = first;
  // The next tile's inputs, as they stand in memory; behind the last tile that one
  // again, behind the last token that one again.
  auto fetch = [&](auto inner, Inputs& in) {
    constexpr bool kInner = decltype(inner)::value;
    uint32_t b_u = o_u, b_d = o_d, b_z = o_z, b_b = o_b, b_c = o_c;
    if (!kInner && ahead + kTile > P.T) {
      const int last = int(P.T - 1 - ahead), t = at < last ? at : last, tb = bc_at < last ? bc_at : last;
      b_u = bytes(t, P.ld_u, c);
      b_d = bytes(t, P.ld_delta, c);
      b_z = bytes(t, P.ld_z, c);
      b_b = bytes(tb, P.ld_b, 0);
      b_c = bytes(tb, P.ld_c, 0);
    }
    load_raw<kWhole>(at_byte(pu, b_u), nc, in.u);
    load_raw<kWhole>(at_byte(pd, b_d), nc, in.delta);
    if constexpr (kGated) load_raw<kWhole>(at_byte(pz, b_z), nc, in.z);
    load_raw<kWhole>(at_byte(pb, b_b), nn, in.Bm);
    if constexpr (!kStates) load_raw<kWhole>(at_byte(pc, b_c), nn, in.Cm);
    if (kInner || ahead + kTile < end) {
      ahead += kTile;
      pu += kTile * P.ld_u, pd += kTile * P.ld_delta, pb += kTile * P.ld_b;
      if constexpr (!kStates) pc += kTile * P.ld_c;
      if constexpr (kGated) pz += kTile * P.ld_z;
    }
  };
  // Converts what was fetched for the tile at t0 and writes its steps.
  auto prepare = [&](auto inner, int64_t t0, int buffer, const Inputs& in, float (&bm)[NS], float (&cm)[NS]) {
    float u[Q], dt[Q], du[Q];
    values(in.u, u);
    values(in.delta, dt);
#pragma unroll
    for (int e = 0; e < Q; ++e) dt[e] += bias[e];
#pragma unroll
    for (int e = 0; e < Q; ++e) {
      const float soft = softplus_f(dt[e]);
      dt[e] = P.softplus ? soft : dt[e];
    }
#pragma unroll
    for (int e = 0; e < Q; ++e) du[e] = dt[e] * u[e];
    values(in.Bm, bm);
    if constexpr (!kStates) values(in.Cm, cm);
    if (!decltype(inner)::value && t0 + kTile > end) {  // behind the end the state stays, whatever stands there
#pragma unroll
      for (int e = 0; e < Q; ++e)
        if (t0 + at >= end) dt[e] = du[e] = 0.0f;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (t0 + bc_at >= end) bm[i] = cm[i] = 0.0f;
    }
    float pair[2 * Q];
#pragma unroll
    for (int e = 0; e < Q; ++e) {
      pair[2 * e] = dt[e];
      pair[2 * e + 1] = du[e];
    }
    __builtin_memcpy(__builtin_assume_aligned(&s_step[buffer][at][lc], Q > 1 ? 16 : 8), pair, 8 * Q);
  };
  // Takes over what was prepared, once the tile before is done with its own.
  float b0[NS], c0[NS];
  auto take = [&](const float (&bm)[NS], const float (&cm)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      b0[i] = bm[i];
      c0[i] = cm[i];
    }
    if (!kStates && shares) {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if (n0 + i >= P.N)
          c0[i] *= part_of;
        else if (kWhole || n0 + i == P.N - 1)
          c0[i] *= rest_of;
      }
    }
  };
  // The waves' shares of y for a thread's token.
  auto collect = [&](int buffer, float (&part)[W][Q]) {
#pragma unroll
    for (int w = 0; w < W; ++w)
      __builtin_memcpy(part[w], __builtin_assume_aligned(&s_y[buffer][kStates ? 0 : w][at][lc], 4 * Q), 4 * Q);
  };
  // y of the tile at t0.
  auto finish = [&](int64_t t0, const float (&part)[W][Q], const Raw<T, Q>& ru, const Raw<T, Q>& rz) {
    float u[Q], z[Q], sum[Q];
    values(ru, u);
#pragma unroll
    for (int e = 0; e < Q; ++e) sum[e] = skip[e] * u[e];
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int e = 0; e < Q; ++e) sum[e] += part[w][e];
    if constexpr (kGated) {
      values(rz, z);
#pragma unroll
      for (int e = 0; e < Q; ++e) sum[e] *= z[e] * logistic_f(z[e]);
    }
    const bool live = t0 >= first && t0 + at < end && lc < p.width;
    T* y = static_cast<T*>(P.y) + (p.b * P.T + t0) * P.D + p.c0;
    if constexpr (kWhole) {
      store_at(y, live ? bytes(at, P.D, c) : kNowhere, sum);
    } else {
      if (live) store_some(at_byte(y, bytes(at, P.D, c)), nc, sum);
    }
  };
  // The sum of the steps (the first wave's), of whole tiles with what rounding lost of them:
  // the steps one after another would drift with the number of tokens (8192 equal ones by more than
  // 1000 x 2^-24), and the decay of many tokens is an exponential of this sum.
  float total = 0.0f, lost = 0.0f;
  Inputs in[2];        // of the next tile and the one after it
  Raw<T, Q> u0{}, z0{}, u1{}, z1{};  // of the present tile and the one before it
  // One tile, at t0: the waves go through it, in[s] is the next one's input.  kInner: the four
  // behind it are whole, and nothing is asked on the way.
  auto tile = [&](auto inner, auto parity, int64_t t0) {
    constexpr int s = decltype(parity)::value;
    float2 step[kTile];
#pragma unroll
    for (int t = 0; t < kTile; ++t) step[t] = s_step[s][t][lane];
    float part[W][Q];
    if constexpr (!kStates) collect(s ^ 1, part);
    __builtin_amdgcn_sched_barrier(0);  // all reads first: a wait for each would follow else
    float bm[NS], cm[NS];
    prepare(inner, t0 + kTile, s ^ 1, in[s], bm, cm);
    const Raw<T, Q> un = in[s].u, zn = in[s].z;
    fetch(inner, in[s]);
    if constexpr (kPass == kMarks) {  // [tile][b][n][D], the steps as one more state
      float* mark = P.marks + (t0 / kTile * P.B + p.b) * (P.N + 1) * P.D + p.c0;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float v[1] = {h[i]};
        store_at(mark + (n0 + i) * P.D, mine && n0 + i < P.N ? uint32_t(lane) * 4 : kNowhere, v);
      }
      const float v[1] = {total};
      store_at(mark + P.N * P.D, mine && wave == 0 ? uint32_t(lane) * 4 : kNowhere, v);
    }
    float steps = 0.0f;  // of this tile
    auto token = [&](auto which) {
      constexpr int t = decltype(which)::value;
      if constexpr (kStates) steps += step[t].x;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        h[i] = fmaf(__builtin_amdgcn_exp2f(step[t].x * a2[i]), h[i],
                    kStates ? row_times<t>(b0[i], step[t].y) : of_row<t>(b0[i]) * step[t].y);
    };
    unrolled<kTile / 2>([&](auto pair) {
      constexpr int t = 2 * decltype(pair)::value;
      float before[NS];
      token(std::integral_constant<int, t>{});
#pragma unroll
      for (int i = 0; i < NS; ++i) before[i] = h[i];
      token(std::integral_constant<int, t + 1>{});
      if constexpr (!kStates) {
        float y0, y1;
        row_dots<t>(c0, before, h, y0, y1);
        s_y[s][wave][t][lane] = y0;
        s_y[s][wave][t + 1][lane] = y1;
      }
      // Two tokens after two: the products of all, made ahead, would not fit the registers.
#pragma unroll
      for (int i = 0; i < NS; ++i) asm volatile("" : "+v"(h[i]));
    });
    if constexpr (kStates) {
      const float more = steps - lost, sum = total + more;
      lost = __builtin_amdgcn_fmed3f((sum - total) - more, -FLT_MAX, FLT_MAX);  // (a number for an infinite sum too)
      total = sum;
    } else {
      finish(t0 - kTile, part, u1, z1);
      u1 = u0, z1 = z0;
      u0 = un, z0 = zn;
    }
    take(bm, cm);
    __syncthreads();
  };
  if (first < end) {
    constexpr std::false_type kAny{};
    constexpr std::true_type kInner{};
    constexpr std::integral_constant<int, 0> kEven{};
    constexpr std::integral_constant<int, 1> kOdd{};
    float bm[NS], cm[NS];
    fetch(kAny, in[1]);
    fetch(kAny, in[0]);
    prepare(kAny, first, 0, in[1], bm, cm);
    take(bm, cm);
    u0 = in[1].u, z0 = in[1].z;
    fetch(kAny, in[1]);
    __syncthreads();
    int64_t t0 = first;
    for (; t0 + 5 * kTile < end; t0 += 2 * kTile) {  // (a token is left to fetch)
      tile(kInner, kEven, t0);
      tile(kInner, kOdd, t0 + kTile);
    }
    for (; t0 + kTile < end; t0 += 2 * kTile) {
      tile(kAny, kEven, t0);
      tile(kAny, kOdd, t0 + kTile);
    }
    const bool odd = t0 < end;
    if (odd) tile(kAny, kEven, t0);
    if constexpr (!kStates) {
      float part[W][Q];
      collect(odd ? 0 : 1, part);
      finish(odd ? t0 : t0 - kTile, part, u1, z1);
    }
  }
  if constexpr (kStates) {
    const int64_t m = (int64_t(p.chunk) * P.B + p.b) * P.N;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (mine && n0 + i < P.N) P.ends[(m + n0 + i) * P.D + d] = h[i];
    if (mine && wave == 0) P.steps[(int64_t(p.chunk) * P.B + p.b) * P.D + d] = total;
  } else {
    // Rows behind the sequence's end are zero.
    const float none[Q] = {};
    for (int64_t t = (first > end ? first : end) + at; t < stop; t += kTile)
      if (lc < p.width) store_some(static_cast<T*>(P.y) + (p.b * P.T + t) * P.D + p.c0 + c, nc, none);
    if (P.h_last != nullptr && stop == P.T) {
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (mine && n0 + i < P.N) P.h_last[(p.b * P.D + d) * P.N + n0 + i] = h[i];
    }
  }
}

// ends[chunk] (what each chunk makes of zero) becomes the state in front of the
// chunk, `reverse` the one behind it when going backwards from `init`; `last`
// receives what comes out at the far end.  One thread per sequence, state and
// channel; the chunks' values are loaded four at a time ahead of the chain.
__global__ __launch_bounds__(256) void carry_kernel(const SelectiveRequest P, const float* init, float* last,
                                                    int reverse) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t bnd = P.B * P.N * P.D;
  if (i >= bnd) return;
  const int64_t d = i % P.D, bn = i / P.D, n = bn % P.N, b = bn / P.N;
  const float a2 = half_rate2(P.A[d * P.N + n]);
  const int64_t own = (b * P.D + d) * P.N + n;
  float h = init ? init[own] : 0.0f;
  constexpr int kAhead = 4;
  for (int c0 = 0; c0 < P.chunks; c0 += kAhead) {
    float e[kAhead], s[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int c = c0 + j < P.chunks ? c0 + j : P.chunks - 1;
      const int64_t k = reverse ? P.chunks - 1 - c : c;
      e[j] = P.ends[k * bnd + i];
      s[j] = P.steps[(k * P.B + b) * P.D + d];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (c0 + j >= P.chunks) break;
      const int64_t k = reverse ? P.chunks - 1 - (c0 + j) : c0 + j;
      P.ends[k * bnd + i] = h;
      // a zero state stays zero however its factor overflows
      h = h == 0.0f ? e[j] : decayed(a2 * s[j], h, e[j]);
    }
  }
  if (last) last[own] = h;
}

// One token: L lanes per channel, V states each, of R streams one after another; y is
// summed over the lanes.  Bound by the states' bytes (read and written once) for
// many streams, whose threads then keep A for four of them, by the launch for a few.
template <typename T, int V, int L, int R>
__global__ __launch_bounds__(256) void step_kernel(const SelectiveRequest P) {
  const int64_t i = int64_t(blockIdx.x) * (256 / L) + threadIdx.x / L;  // streams' group and channel
  const int n0 = threadIdx.x % L * V;
  const int64_t groups = (P.B + R - 1) / R;
  const bool live = i < groups * P.D;
  const int64_t k = live ? i : groups * P.D - 1;
  const int64_t b0 = k / P.D * R, d = k % P.D, g0 = d / (P.D / P.G) * P.N;
  const bool has = n0 < P.N;
  const int n = has ? n0 : 0;
  // states n .. n + V - 1 (with V = 4, N is a multiple of four)
  auto load_states = [&](const auto* p, float (&v)[V]) {
    if constexpr (V == 4)
      load_n(p, v);
    else
      v[0] = to_f32(*p);
  };
  float a[V], h[R][V], bm[R][V], cm[R][V], u[R], x[R], z[R];
  load_states(P.A + d * P.N + n, a);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t b = b0 + r < P.B ? b0 + r : P.B - 1;
    if (P.h0) {
      load_states(P.h0 + (b * P.D + d) * P.N + n, h[r]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) h[r][v] = 0.0f;
    }
    load_states(static_cast<const T*>(P.Bm) + b * P.ld_b + g0 + n, bm[r]);
    load_states(static_cast<const T*>(P.Cm) + b * P.ld_c + g0 + n, cm[r]);
    u[r] = to_f32(static_cast<const T*>(P.u)[b * P.ld_u + d]);
    x[r] = to_f32(static_cast<const T*>(P.delta)[b * P.ld_delta + d]);
    z[r] = P.z ? to_f32(static_cast<const T*>(P.z)[b * P.ld_z + d]) : 0.0f;
  }
  const float skip = P.skip ? P.skip[d] : 0.0f, bias = P.bias ? P.bias[d] : 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float soft = softplus_f(x[r] + bias);
    const float dt = P.softplus ? soft : x[r] + bias;
    const float du = dt * u[r];
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[r][v] = fmaf(__builtin_amdgcn_exp2f(dt * rate2(a[v])), h[r][v], du * bm[r][v]);
      sum = has ? fmaf(h[r][v], cm[r][v], sum) : 0.0f;
    }
#pragma unroll
    for (int m = 1; m < L; m *= 2) sum += __shfl_xor(sum, m);
    const int64_t b = b0 + r;
    if (!live || b >= P.B) continue;
    if (has) {
      float* to = P.h_last + (b * P.D + d) * P.N + n;
      if constexpr (V == 4)
        store_n(to, h[r]);
      else
        *to = h[r][0];
    }
    if (n0 == 0) {
      sum = fmaf(skip, u[r], sum);
      if (P.z) sum *= z[r] * logistic_f(z[r]);
      static_cast<T*>(P.y)[b * P.D + d] = from_f32<T>(sum);
    }
  }
}

template <typename T, int W, int NS, int kPass, bool kGated = false>
void launch_pass(const SelectiveRequest& P, uint32_t blocks) {
  constexpr int Q = kTile / W;
  const bool whole =
      P.D / P.G % Q == 0 && P.N % NS == 0 && reinterpret_cast<uintptr_t>(P.y) % (Q * sizeof(T)) == 0;
  auto run = [&](auto* kernel) { hipLaunchKernelGGL(kernel, dim3(blocks), dim3(W * 64), 0, P.stream, P); };
  if (whole)
    run(scan_kernel<T, W, NS, kPass, true, kGated>);
  else
    run(scan_kernel<T, W, NS, kPass, false, kGated>);
}
template <typename T, int W, int NS>
void launch_scan(const SelectiveRequest& P, int pass, uint32_t blocks) {
  if (pass == kEnds)
    launch_pass<T, W, NS, kEnds>(P, blocks);
  else if (pass == kMarks)
    launch_pass<T, W, NS, kMarks>(P, blocks);
  else if (P.z)
    launch_pass<T, W, NS, kOutputs, true>(P, blocks);
  else
    launch_pass<T, W, NS, kOutputs, false>(P, blocks);
}
template <typename T>
void launch_scan(const SelectiveRequest& P, int pass, uint32_t blocks) {
  if (P.N <= 4)
    launch_scan<T, 4, 1>(P, pass, blocks);
  else if (P.N <= 8)
    launch_scan<T, 4, 2>(P, pass, blocks);
  else if (P.N <= 16)
    launch_scan<T, 4, 4>(P, pass, blocks);
  else if (P.N <= 32)
    launch_scan<T, 8, 4>(P, pass, blocks);
  else
    launch_scan<T, 8, 8>(P, pass, blocks);
}

// Of a step: states per lane, lanes per channel, streams per thread.
struct StepShape {
  int states, lanes, streams;
};
StepShape step_shape(int64_t B, int64_t D, int64_t N) {
  StepShape s{N % 4 == 0 ? 4 : 1, 1, 1};
  while (s.lanes * s.states < N) s.lanes *= 2;
  // Four streams per thread where that leaves two waves per SIMD.  Measured in us, D = 2048,
  // 16 states, one stream / four: 32 streams 4.1 / 4.7, 64 6.0 / 5.9, 128 9.6 / 8.4, 1024 51.6 / 46.2.
  if (B / 4 * D * s.lanes >= 2 * 4 * 256 * 64) s.streams = 4;
  return s;
}

template <typename T, int V, int L>
void launch_step(const SelectiveRequest& P, int streams) {
  const dim3 blocks(uint32_t(selective_step_blocks(P.B, P.D, P.N)));
  if (streams == 4)
    hipLaunchKernelGGL((step_kernel<T, V, L, 4>), blocks, dim3(256), 0, P.stream, P);
  else
    hipLaunchKernelGGL((step_kernel<T, V, L, 1>), blocks, dim3(256), 0, P.stream, P);
}
template <typename T, int V>
void launch_step(const SelectiveRequest& P, StepShape shape) {
  switch (shape.lanes) {
    case 1: return launch_step<T, V, 1>(P, shape.streams);
    case 2: return launch_step<T, V, 2>(P, shape.streams);
    case 4: return launch_step<T, V, 4>(P, shape.streams);
    case 8: return launch_step<T, V, 8>(P, shape.streams);
    case 16: return launch_step<T, V, 16>(P, shape.streams);
  }
  if constexpr (V == 1) {
    if (shape.lanes == 32)
      launch_step<T, V, 32>(P, shape.streams);
    else
      launch_step<T, V, 64>(P, shape.streams);
  }
}

sr_status launched(const char* what) {
  const hipError_t err = hipGetLastError();
  return err == hipSuccess ? SR_OK : fail(SR_ERR_HIP, "%s: %s", what, hipGetErrorString(err));
}

}  // namespace

namespace {

// The plan with about `want` chunks: none below 128 tokens, whose two more launches
// would cost what they save, nor shorter than 2 sqrt(T) tokens, so that the carry over
// the chunks stays as short as the walk through one.
SelectivePlan chunked(int64_t T, int64_t tiles_per_group, int64_t want) {
  SelectivePlan plan{tiles_per_group, 1, T};
  if (T < kSelectiveMinTokens) return plan;
  int64_t shortest = kTile;
  while (shortest * shortest < 4 * T) shortest += kTile;
  const int64_t most = T / shortest;
  if (want > most) want = most;
  if (want > 1) {
    plan.chunk_len = ((T + want - 1) / want + kTile - 1) / kTile * kTile;
    plan.chunks = (T + plan.chunk_len - 1) / plan.chunk_len;
  }
  return plan;
}

}  // namespace

// Chunks over time: none where sequences and channels fill the GPU by themselves (the
// first pass computes three quarters of what the second does), else about 1536 workgroups
// in all.  Measured, 4096 tokens in bf16, workgroups without chunks: us without chunks /
// with them: 8: 353 / 37, 64: 354 / 131, 128: 349 / 242, 192: 351 / 344, 256: 356 / 455.
// In all 256 / 512 / 1024 / 1536 / 2048 of them, us: 1 x 65536 x 1024 with 4 states 380 / 272 / 251 / 247 / 252,
// 16 states 601 / 498 / 467 / 465 / 463, 64 states 1528 / 1498 / 1504 / 1527 / 1543; 4 x 4096 x 2048 with 4 states
// 179 / 136 / 123 / 124 / 122, 16 states 306 / 256 / 239 / 241 / 236, 64 states 778 / 764 / 775 / 806 / 805.
SelectivePlan selective_plan(int64_t B, int64_t T, int64_t D, int64_t G) {
  const int64_t tiles = (D / G + kLanes - 1) / kLanes, blocks = B * G * tiles;
  return chunked(T, tiles, blocks > 0 && blocks < 224 ? (1536 + blocks - 1) / blocks : 1);
}

// The backward pass has one workgroup per CU at a time, and its chunks cost a fifth more
// (the pass that carries gradients backwards): the number of them that leaves the
// fewest rounds over the 256 CUs for a chunk's work, where a round's start and end cost 0.15 of it and a
// chunk's carry 0.002.  Measured in us, 2048 tokens, 16 states, workgroups without chunks: without / the rule's / the
// best of 2 to 32 chunks: 8: 698 / 86 / 83, 64: 710 / 250 / 242, 128: 721 / 459 / 441, 192: 730 / 657 / 642,
// 256: 736 / 736 / 832, 320: 1372 / 1058 / 1032, 640: 2049 / 2118 / 1993; 8192 tokens, 16 workgroups 2750 / 250 / 246.
SelectivePlan selective_backward_plan(int64_t B, int64_t T, int64_t D, int64_t G) {
  const int64_t tiles = (D / G + kLanes - 1) / kLanes, blocks = B * G * tiles;
  int64_t best = 1;
  double least = 0.15 + double((blocks + 255) / 256);
  for (int64_t k = 2; k <= 64 && blocks > 0 && blocks < 1024; ++k) {
    const double cost = 1.2 * (0.15 + double((blocks * k + 255) / 256)) / double(k) + 0.002 * double(k);
    if (cost < least) {
      least = cost;
      best = k;
    }
  }
  return chunked(T, tiles, best);
}

sr_status launch_selective_states(const SelectiveRequest& P) {
  const uint32_t blocks = uint32_t(P.B * P.G * P.tiles_per_group * P.chunks);
  if (P.dtype == SR_BF16)
    launch_scan<uint16_t>(P, P.marks ? kMarks : kEnds, blocks);
  else
    launch_scan<float>(P, P.marks ? kMarks : kEnds, blocks);
  return launched("selective scan states");
}

sr_status launch_selective_carry(const SelectiveRequest& P, const float* init, float* last, bool reverse) {
  const int64_t n = P.B * P.N * P.D;
  hipLaunchKernelGGL(carry_kernel, dim3(uint32_t((n + 255) / 256)), dim3(256), 0, P.stream, P, init, last,
                     int(reverse));
  return launched("selective scan carry");
}

sr_status launch_selective_scan(const SelectiveRequest& rq) {
  SelectiveRequest P = rq;
  if (P.chunks > 1) {
    sr_status st = launch_selective_states(P);
    if (st != SR_OK) return st;
    st = launch_selective_carry(P, P.h0, nullptr, false);
    if (st != SR_OK) return st;
  } else {
    P.ends = nullptr;
  }
  const uint32_t blocks = uint32_t(P.B * P.G * P.tiles_per_group * P.chunks);
  if (P.dtype == SR_BF16)
    launch_scan<uint16_t>(P, kOutputs, blocks);
  else
    launch_scan<float>(P, kOutputs, blocks);
  return launched("selective scan");
}

int64_t selective_step_blocks(int64_t B, int64_t D, int64_t N) {
  const StepShape s = step_shape(B, D, N);
  const int64_t per = 256 / s.lanes;
  return ((B + s.streams - 1) / s.streams * D + per - 1) / per;
}

sr_status launch_selective_step(const SelectiveRequest& P) {
  const bool bf16 = P.dtype == SR_BF16;
  const StepShape shape = step_shape(P.B, P.D, P.N);
  if (shape.states == 4) {
    if (bf16)
      launch_step<uint16_t, 4>(P, shape);
    else
      launch_step<float, 4>(P, shape);
  } else {
    if (bf16)
      launch_step<uint16_t, 1>(P, shape);
    else
      launch_step<float, 1>(P, shape);
  }
  return launched("selective step");
}

}  // namespace sr
