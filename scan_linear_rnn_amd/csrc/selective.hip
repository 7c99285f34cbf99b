// The selective state space scan over a sequence, and its single-token step.
//
//     dt = softplus(delta + bias)                      (or delta + bias)
//     h_n <- exp(dt A_n) h_n + (dt u) B_n              n = 1..N, per channel
//     y  = (sum_n C_n h_n + skip u) silu(z)
//
// with A per channel and state, and B, C per token (shared by the channels of
// a group).  States, sums and gates are fp32; y is rounded once.
//
// A workgroup owns 64 channels (a lane each) of one sequence and walks over
// its tokens in tiles of 16; its waves hold four states per lane each.  The
// waves share what is per token and channel: each prepares a part of the
// tile's steps (softplus and the like) in LDS, and sums its part of the
// waves' shares of y.  So every input is read once, wide, and the
// recurrence, 16 x (2 products, exp, 2 fused multiply-adds), is what the
// vector units spend their time on.
//
// Where there are too few sequences and channels to fill the GPU, the tokens are
// cut into chunks: a first pass (kStates) computes what each chunk adds to a
// zero state and the sum of its steps, whose exponential is the chunk's decay; one
// thread per state then carries the states over the chunks (carry_kernel); and the
// full pass starts each chunk from its own state.

#include "layer_util.hpp"

namespace sr {
namespace {

// kStates: the state that the chunk's tokens make of zero (P.ends) and the sum
// of their steps (P.steps), and with P.marks what the chunk has made of zero in
// front of each tile, with the sum of the steps so far.  Else: y from the chunk's own
// start state, and the last state.
template <typename T, int W, bool kStates>
__global__ __launch_bounds__(W * 64) void scan_kernel(const SelectiveRequest P) {
  constexpr int kSlots = kTile * kLanes / 4;                    // four channels of one token each
  constexpr int kPer = kSlots > W * 64 ? kSlots / (W * 64) : 1;  // a thread's
  constexpr int kN = W * kNS;
  __shared__ __align__(16) float2 s_step[kTile][kLanes];  // dt, dt u
  __shared__ float s_b[kTile][kN], s_c[kStates ? 1 : kTile][kN];
  __shared__ __align__(16) float s_y[kStates ? 1 : W][kTile][kLanes];
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
  const T* Bm = static_cast<const T*>(P.Bm);
  const T* Cm = static_cast<const T*>(P.Cm);
  T* y = static_cast<T*>(P.y);

  const int64_t d = p.c0 + lane;
  const int n0 = wave * kNS;
  const bool mine = lane < p.width;
  float a2[kNS], h[kNS];
#pragma unroll
  for (int i = 0; i < kNS; ++i) {
    const bool is = mine && n0 + i < P.N;
    a2[i] = is ? P.A[d * P.N + n0 + i] * kLog2e : 0.0f;
    h[i] = 0.0f;
    if constexpr (!kStates) {
      if (P.ends != nullptr) {  // [chunk][b][n][D]
        if (is) h[i] = P.ends[((int64_t(p.chunk) * P.B + p.b) * P.N + n0 + i) * P.D + d];
      } else if (P.h0 != nullptr && is) {
        h[i] = P.h0[(p.b * P.D + d) * P.N + n0 + i];
      }
    }
  }

  int at[kPer], c4[kPer];  // a slot's token in the tile and first channel
  f32x4 bias[kPer], skip[kPer], ru[kPer], rd[kPer], rz[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int slot = tid + j * W * 64;
    at[j] = slot / (kLanes / 4);
    c4[j] = slot % (kLanes / 4) * 4;
    if (slot >= kSlots || c4[j] >= p.width) at[j] = kTile;  // nothing to do
    bias[j] = skip[j] = rz[j] = f32x4{};
    if (at[j] < kTile) {
      const int n = p.width - c4[j];
      if (P.bias) bias[j] = load4(P.bias + p.c0 + c4[j], n);
      if (!kStates && P.skip) skip[j] = load4(P.skip + p.c0 + c4[j], n);
    }
  }
  // The inputs of the slots of the tile at t0; zeros behind the end.
  auto fetch = [&](int64_t t0) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      ru[j] = rd[j] = f32x4{};
      if (at[j] < kTile && t0 + at[j] < end) {
        const int64_t row = p.b * P.T + t0 + at[j], c = p.c0 + c4[j];
        const int n = p.width - c4[j];
        ru[j] = load4(u + row * P.ld_u + c, n);
        rd[j] = load4(delta + row * P.ld_delta + c, n);
        if (!kStates && z) rz[j] = load4(z + row * P.ld_z + c, n);
      }
    }
  };
  float total = 0.0f;  // of the steps (the first wave's)
  fetch(first);
  for (int64_t t0 = first; t0 < end; t0 += kTile) {
    f32x4 cu[kPer], cz[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      cu[j] = ru[j];
      cz[j] = rz[j];
      if (at[j] >= kTile) continue;
      f32x4 dt = rd[j] + bias[j];
      if (P.softplus) {
#pragma unroll
        for (int e = 0; e < 4; ++e) dt[e] = softplus_f(dt[e]);
      }
      const f32x4 du = dt * cu[j];
      f32x4* to = reinterpret_cast<f32x4*>(&s_step[at[j]][c4[j]]);
      to[0] = f32x4{dt[0], du[0], dt[1], du[1]};
      to[1] = f32x4{dt[2], du[2], dt[3], du[3]};
    }
    for (int i = tid; i < kTile * kN; i += W * 64) {
      const int t = i / kN, n = i % kN;
      const bool is = t0 + t < end && n < P.N;
      const int64_t row = p.b * P.T + t0 + t, off = int64_t(p.group) * P.N + n;
      s_b[t][n] = is ? to_f32(Bm[row * P.ld_b + off]) : 0.0f;
      if constexpr (!kStates) s_c[t][n] = is ? to_f32(Cm[row * P.ld_c + off]) : 0.0f;
    }
    fetch(t0 + kTile);
    __syncthreads();
    if constexpr (kStates) {
      if (P.marks != nullptr) {  // [tile][b][n][D], the steps as one more state
        const int64_t m = (t0 / kTile * P.B + p.b) * (P.N + 1);
#pragma unroll
        for (int i = 0; i < kNS; ++i)
          if (mine && n0 + i < P.N) P.marks[(m + n0 + i) * P.D + d] = h[i];
        if (mine && wave == 0) P.marks[(m + P.N) * P.D + d] = total;
      }
    }
    const int count = int(end - t0 < kTile ? end - t0 : kTile);
    auto step = [&](int t) {
      const float2 s = s_step[t][lane];
      total += s.x;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kNS; ++i) {
        h[i] = fmaf(__builtin_amdgcn_exp2f(s.x * a2[i]), h[i], s.y * s_b[t][n0 + i]);
        if constexpr (!kStates) sum = fmaf(h[i], s_c[t][n0 + i], sum);
      }
      if constexpr (!kStates) s_y[wave][t][lane] = sum;
    };
    if (count == kTile) {
#pragma unroll
      for (int t = 0; t < kTile; ++t) step(t);
    } else {
      for (int t = 0; t < count; ++t) step(t);
    }
    __syncthreads();
    if constexpr (!kStates) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (at[j] >= count) continue;
        f32x4 sum = skip[j] * cu[j];
#pragma unroll
        for (int w = 0; w < W; ++w) sum += *reinterpret_cast<const f32x4*>(&s_y[w][at[j]][c4[j]]);
        if (z) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] *= cz[j][e] * logistic_f(cz[j][e]);
        }
        store4(y + (p.b * P.T + t0 + at[j]) * P.D + p.c0 + c4[j], sum, p.width - c4[j]);
      }
    }
  }
  if constexpr (kStates) {
    const int64_t m = (int64_t(p.chunk) * P.B + p.b) * P.N;
#pragma unroll
    for (int i = 0; i < kNS; ++i)
      if (mine && n0 + i < P.N) P.ends[(m + n0 + i) * P.D + d] = h[i];
    if (mine && wave == 0) P.steps[(int64_t(p.chunk) * P.B + p.b) * P.D + d] = total;
  } else {
    // Rows behind the sequence's end are zero.
    for (int64_t t0 = first > end ? first : end; t0 < stop; t0 += kTile) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (at[j] < kTile && t0 + at[j] < stop)
          store4(y + (p.b * P.T + t0 + at[j]) * P.D + p.c0 + c4[j], f32x4{}, p.width - c4[j]);
    }
    if (P.h_last != nullptr && stop == P.T) {
#pragma unroll
      for (int i = 0; i < kNS; ++i)
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
  const float a2 = P.A[d * P.N + n] * kLog2e;
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
      h = h == 0.0f ? e[j] : fmaf(__builtin_amdgcn_exp2f(a2 * s[j]), h, e[j]);
    }
  }
  if (last) last[own] = h;
}

// One token: L lanes per channel, V states each; y is summed over the lanes.
// Bound by the states' bytes (read and written once) for many streams, by the
// launch for a few.
template <typename T, int V, int L>
__global__ __launch_bounds__(256) void step_kernel(const SelectiveRequest P) {
  const int64_t i = int64_t(blockIdx.x) * (256 / L) + threadIdx.x / L;  // row and channel
  const int n0 = threadIdx.x % L * V;
  const bool live = i < P.B * P.D;
  const int64_t k = live ? i : P.B * P.D - 1;
  const int64_t b = k / P.D, d = k - b * P.D;
  const T* Bm = static_cast<const T*>(P.Bm) + b * P.ld_b + d / (P.D / P.G) * P.N;
  const T* Cm = static_cast<const T*>(P.Cm) + b * P.ld_c + d / (P.D / P.G) * P.N;
  float h[V], a[V], bm[V], cm[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = a[v] = bm[v] = cm[v] = 0.0f;
  if (n0 < P.N) {
    if constexpr (V == 4) {  // N is a multiple of four
      const f32x4 av = load4(P.A + d * P.N + n0, 4), bv = load4(Bm + n0, 4), cv = load4(Cm + n0, 4);
      f32x4 hv{};
      if (P.h0) hv = load4(P.h0 + k * P.N + n0, 4);
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = hv[v], a[v] = av[v], bm[v] = bv[v], cm[v] = cv[v];
    } else {
      if (P.h0) h[0] = P.h0[k * P.N + n0];
      a[0] = P.A[d * P.N + n0];
      bm[0] = to_f32(Bm[n0]);
      cm[0] = to_f32(Cm[n0]);
    }
  }
  const float u = to_f32(static_cast<const T*>(P.u)[b * P.ld_u + d]);
  float x = to_f32(static_cast<const T*>(P.delta)[b * P.ld_delta + d]);
  const float zv = P.z ? to_f32(static_cast<const T*>(P.z)[b * P.ld_z + d]) : 0.0f;
  const float skip = P.skip ? P.skip[d] : 0.0f;
  if (P.bias) x += P.bias[d];
  const float dt = P.softplus ? softplus_f(x) : x;
  const float du = dt * u;
  float sum = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = fmaf(__builtin_amdgcn_exp2f(dt * (a[v] * kLog2e)), h[v], du * bm[v]);
    sum = fmaf(h[v], cm[v], sum);
  }
  if (live && n0 < P.N) {
    if constexpr (V == 4)
      store4(P.h_last + i * P.N + n0, f32x4{h[0], h[1], h[2], h[3]}, 4);
    else
      P.h_last[i * P.N + n0] = h[0];
  }
#pragma unroll
  for (int m = 1; m < L; m *= 2) sum += __shfl_xor(sum, m);
  if (live && n0 == 0) {
    sum = fmaf(skip, u, sum);
    if (P.z) sum *= zv * logistic_f(zv);
    static_cast<T*>(P.y)[i] = from_f32<T>(sum);
  }
}

template <typename T, int W>
void launch_scan(const SelectiveRequest& P, bool states, uint32_t blocks) {
  if (states)
    hipLaunchKernelGGL((scan_kernel<T, W, true>), dim3(blocks), dim3(W * 64), 0, P.stream, P);
  else
    hipLaunchKernelGGL((scan_kernel<T, W, false>), dim3(blocks), dim3(W * 64), 0, P.stream, P);
}
template <typename T>
void launch_scan(const SelectiveRequest& P, bool states, uint32_t blocks) {
  if (P.N <= 4)
    launch_scan<T, 1>(P, states, blocks);
  else if (P.N <= 8)
    launch_scan<T, 2>(P, states, blocks);
  else if (P.N <= 16)
    launch_scan<T, 4>(P, states, blocks);
  else if (P.N <= 32)
    launch_scan<T, 8>(P, states, blocks);
  else
    launch_scan<T, 16>(P, states, blocks);
}

template <typename T, int V>
void launch_step(const SelectiveRequest& P) {
  const int64_t lanes = (P.N + V - 1) / V;
  auto run = [&](auto* kernel, int L) {
    const int64_t blocks = (P.B * P.D + 256 / L - 1) / (256 / L);
    hipLaunchKernelGGL(kernel, dim3(uint32_t(blocks)), dim3(256), 0, P.stream, P);
  };
  if (lanes <= 1)
    run(step_kernel<T, V, 1>, 1);
  else if (lanes <= 2)
    run(step_kernel<T, V, 2>, 2);
  else if (lanes <= 4)
    run(step_kernel<T, V, 4>, 4);
  else if (lanes <= 8)
    run(step_kernel<T, V, 8>, 8);
  else if (lanes <= 16)
    run(step_kernel<T, V, 16>, 16);
  else if constexpr (V == 1) {
    if (lanes <= 32)
      run(step_kernel<T, V, 32>, 32);
    else
      run(step_kernel<T, V, 64>, 64);
  }
}

sr_status launched(const char* what) {
  const hipError_t err = hipGetLastError();
  return err == hipSuccess ? SR_OK : fail(SR_ERR_HIP, "%s: %s", what, hipGetErrorString(err));
}

}  // namespace

// Chunks over time: none where sequences and channels fill the GPU by
// themselves (the first pass computes nearly as much as the second), else
// enough of them for a few workgroups per CU.
SelectivePlan selective_plan(int64_t B, int64_t T, int64_t D, int64_t G) {
  SelectivePlan plan{};
  const int64_t per = G ? D / G : 0;
  plan.tiles_per_group = (per + kLanes - 1) / kLanes;
  const int64_t blocks = B * G * plan.tiles_per_group;
  plan.chunks = 1;
  plan.chunk_len = T;
  if (blocks > 0 && blocks < 192 && T >= 2 * kSelectiveMinChunk) {
    int64_t want = (1024 + blocks - 1) / blocks;
    const int64_t most = T / kSelectiveMinChunk;
    if (want > most) want = most;
    plan.chunk_len = ((T + want - 1) / want + kTile - 1) / kTile * kTile;
    plan.chunks = (T + plan.chunk_len - 1) / plan.chunk_len;
  }
  return plan;
}

SelectivePlan selective_backward_plan(int64_t B, int64_t T, int64_t D, int64_t G) {
  return selective_plan(B, T, D, G);
}

sr_status launch_selective_states(const SelectiveRequest& P) {
  const uint32_t blocks = uint32_t(P.B * P.G * P.tiles_per_group * P.chunks);
  if (P.dtype == SR_BF16)
    launch_scan<uint16_t>(P, true, blocks);
  else
    launch_scan<float>(P, true, blocks);
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
    launch_scan<uint16_t>(P, false, blocks);
  else
    launch_scan<float>(P, false, blocks);
  return launched("selective scan");
}

sr_status launch_selective_step(const SelectiveRequest& P) {
  const bool bf16 = P.dtype == SR_BF16;
  if (P.N % 4 == 0) {
    if (bf16)
      launch_step<uint16_t, 4>(P);
    else
      launch_step<float, 4>(P);
  } else {
    if (bf16)
      launch_step<uint16_t, 1>(P);
    else
      launch_step<float, 1>(P);
  }
  return launched("selective step");
}

}  // namespace sr
