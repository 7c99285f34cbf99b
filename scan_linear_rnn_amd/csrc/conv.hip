// The short causal convolution over a sequence, a filter of K taps per channel:
//
//     c_t = bias + sum_j w_j x_{t-K+1+j},   y_t = silu(c_t)  (or c_t)
//
// with the last K - 1 inputs as the state that a following call takes in front of
// its tokens.  Bound by the bytes of x and y: 8 x 4096 x 2048 in bf16 takes 46 us, 5.8
// TB/s; its single-token form, 256 x 2048, 4.1 us (the call 5.1, bound by the host).  A thread owns 16 bytes of
// channels and a run of tokens, keeps the window of its taps in registers and reads
// every input once but for the K - 1 in front of its run; the next tokens' loads
// are on the way while the present ones are computed.  Where D is no multiple
// of a thread's channels, the last thread of a row starts so that it ends with
// the row: it repeats some of its neighbour's channels, with the same results.

#include "layer_util.hpp"

namespace sr {
namespace {

constexpr int kAhead = 4;  // tokens loaded at a time

struct Run {
  int64_t b, t0, t1, c, length;  // tokens [t0, t1) of sequence b, first channel, the sequence's tokens
  int64_t index;                 // of all runs
};
template <int V>
__device__ __forceinline__ bool run_of(const ConvRequest& P, int64_t i, Run* r) {
  const int64_t nvec = (P.D + V - 1) / V;
  const int64_t c = i % nvec * V;
  r->index = i / nvec;
  r->b = r->index / P.runs;
  if (r->b >= P.B) return false;
  r->c = c + V <= P.D ? c : P.D - V;
  r->t0 = r->index % P.runs * P.run_len;
  r->t1 = r->t0 + P.run_len < P.T ? r->t0 + P.run_len : P.T;
  r->length = P.T;
  if (P.lengths) {
    const int64_t n = P.lengths[r->b];
    r->length = n < 0 ? 0 : n < P.T ? n : P.T;
  }
  return true;
}

// V elements, an odd number of them one by one.
template <int V, typename T>
__device__ __forceinline__ void load_v(const T* p, float (&v)[V]) {
  if constexpr (V % 2) {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = to_f32(p[e]);
  } else {
    load_n(p, v);
  }
}
template <int V, typename T>
__device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
  if constexpr (V == 1)
    *p = from_f32<T>(v[0]);
  else
    store_n(p, v);
}

// The input at token t of the sequence: from x, or in front of it from the
// state, or zero.
template <typename T, int K, int V>
__device__ __forceinline__ void input_at(const ConvRequest& P, int64_t b, int64_t t, int64_t c, float (&v)[V]) {
  if (t >= 0) {
    load_v(static_cast<const T*>(P.x) + (b * P.T + t) * P.ld_x + c, v);
  } else if (P.state) {
    load_v(static_cast<const T*>(P.state) + (b * (K - 1) + K - 1 + t) * P.D + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0.0f;
  }
}

// The filters of V neighbouring channels stand one after another.
template <int K, int V, typename W>
__device__ __forceinline__ void load_taps(const W* w0, const W* b0, int64_t c, float (&w)[K][V], float (&bias)[V]) {
  float all[V * K];
  load_v(w0 + c * K, all);
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][e] = all[e * K + j];
    bias[e] = 0.0f;
  }
  if (b0) load_v(b0 + c, bias);
}
template <int K, int V>
__device__ __forceinline__ void load_taps(const ConvRequest& P, int64_t c, float (&w)[K][V], float (&bias)[V]) {
  if (P.w_dtype == SR_BF16)
    load_taps<K, V>(static_cast<const uint16_t*>(P.w), static_cast<const uint16_t*>(P.bias), c, w, bias);
  else
    load_taps<K, V>(static_cast<const float*>(P.w), static_cast<const float*>(P.bias), c, w, bias);
}

template <typename T, int K, int V>
__global__ __launch_bounds__(256) void conv_kernel(const ConvRequest P) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t nvec = (P.D + V - 1) / V, main = P.B * P.runs * nvec;
  if (i >= main) {  // the state behind each sequence
    const int64_t k = i - main, rest = k / nvec;
    if (P.last == nullptr || rest >= P.B * (K - 1)) return;
    constexpr int kKept = K > 1 ? K - 1 : 1;
    const int64_t b = rest / kKept, m = rest % kKept;
    const int64_t c = k % nvec * V + V <= P.D ? k % nvec * V : P.D - V;
    int64_t length = P.T;
    if (P.lengths) {
      const int64_t n = P.lengths[b];
      length = n < 0 ? 0 : n < P.T ? n : P.T;
    }
    float v[V];
    input_at<T, K>(P, b, length - (K - 1) + m, c, v);
    store_v(static_cast<T*>(P.last) + (b * (K - 1) + m) * P.D + c, v);
    return;
  }
  Run r;
  if (!run_of<V>(P, i, &r)) return;
  float w[K][V], bias[V], win[K][V];  // win[j]: the input under tap j
  load_taps<K>(P, r.c, w, bias);
  const T* x = static_cast<const T*>(P.x) + r.b * P.T * P.ld_x + r.c;
  T* y = static_cast<T*>(P.y) + r.b * P.T * P.D + r.c;
  const int64_t end = r.length < r.t1 ? r.length : r.t1;
  if (r.t0 < end) {
#pragma unroll
    for (int j = 1; j < K; ++j) input_at<T, K>(P, r.b, r.t0 - K + j, r.c, win[j]);
  }
  auto token = [&](int64_t t, const Raw<T, V>& in) {
    float x1[V], out[V];
    values(in, x1);
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int j = 0; j + 1 < K; ++j) win[j][e] = win[j + 1][e];
      win[K - 1][e] = x1[e];
      float c = bias[e];
#pragma unroll
      for (int j = 0; j < K; ++j) c = fmaf(w[j][e], win[j][e], c);
      out[e] = P.silu ? c * logistic_f(c) : c;
    }
    store_v(y + t * P.D, out);
  };
  // Whole groups of tokens without a condition (a store that may not happen would
  // have the loads behind it wait for all stores), then what is left.
  int64_t t = r.t0;
  if (t + kAhead <= end) {
    Raw<T, V> next[kAhead];
    auto fetch = [&](int64_t t1) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) load_raw<true>(x + (t1 + a < end ? t1 + a : end - 1) * P.ld_x, V, next[a]);
    };
    fetch(t);
    for (; t + kAhead <= end; t += kAhead) {
      Raw<T, V> in[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) in[a] = next[a];
      fetch(t + kAhead);
#pragma unroll
      for (int a = 0; a < kAhead; ++a) token(t + a, in[a]);
    }
  }
  for (; t < end; ++t) {
    Raw<T, V> in;
    load_raw<true>(x + t * P.ld_x, V, in);
    token(t, in);
  }
  // Rows behind the sequence's end are zero.
  const float none[V] = {};
  for (t = end > r.t0 ? end : r.t0; t < r.t1; ++t) store_v(y + t * P.D, none);
}

// Backward.  With dc_t = dy_t silu'(c_t):
//     dx_s = sum_j w_j dc_{s+K-1-j},  dw_j = sum_t dc_t x_{t-K+1+j},  dbias = sum_t dc_t
// and the gradient of the state behind the sequence added to the inputs it is made of.
// A run goes over its tokens and the K - 1 behind it (whose dc it computes too), so
// dx needs no second pass (8 x 2048 x 1024 in bf16 27 us, 3.7 TB/s: one wave per
// SIMD, its vector unit active for two thirds of the time; shorter runs and two waves take as
// long, and about 64 bytes per lane are on their way); a run's sums for dw and dbias go out per run and are added
// up by column_sums.
template <typename T, int K, int V>
__global__ __launch_bounds__(256) void conv_backward_kernel(const ConvRequest P) {
  Run r;
  if (!run_of<V>(P, int64_t(blockIdx.x) * 256 + threadIdx.x, &r)) return;
  float w[K][V], bias[V], win[K][V], dc[K][V], dw[K][V], dbias[V];  // dc[j]: of the token j before the present one
  load_taps<K>(P, r.c, w, bias);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    dbias[e] = 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][e] = dc[j][e] = win[j][e] = 0.0f;
  }
  const T* x = static_cast<const T*>(P.x) + r.b * P.T * P.ld_x + r.c;
  const T* dy = static_cast<const T*>(P.dy) + r.b * P.T * P.ld_dy + r.c;
  T* dx = static_cast<T*>(P.dx) + r.b * P.T * P.D + r.c;
  const int64_t stop = r.t1 + K - 1;
  const int64_t end = r.length < stop ? r.length : stop;  // tokens from here on give nothing
  if (r.t0 < end) {
#pragma unroll
    for (int j = 1; j < K; ++j) input_at<T, K>(P, r.b, r.t0 - K + j, r.c, win[j]);
  }
  // One token: kInside, all of its parts exist and its neighbours' do.
  auto token = [&](auto inside, int64_t t, const Raw<T, V>& in_x, const Raw<T, V>& in_g) {
    constexpr bool kInside = decltype(inside)::value;
    const bool live = kInside || t < end, own = kInside || t < r.t1;
    float x1[V], g1[V], out[V];
    values(in_x, x1);
    values(in_g, g1);
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int j = 0; j + 1 < K; ++j) win[j][e] = win[j + 1][e];
      win[K - 1][e] = live ? x1[e] : 0.0f;
#pragma unroll
      for (int j = K - 1; j > 0; --j) dc[j][e] = dc[j - 1][e];
      float g = g1[e];
      float c = bias[e];
#pragma unroll
      for (int j = 0; j < K; ++j) c = fmaf(w[j][e], win[j][e], c);
      const float s = logistic_f(c), slope = s * fmaf(c, 1.0f - s, 1.0f);
      g *= P.silu ? slope : 1.0f;
      dc[0][e] = live ? g : 0.0f;
      // (not a product with zero for the other tokens: an input in their window may be infinite)
      const bool counts = live && own;
      dbias[e] += counts ? dc[0][e] : 0.0f;
#pragma unroll
      for (int j = 0; j < K; ++j) dw[j][e] = counts ? fmaf(dc[0][e], win[j][e], dw[j][e]) : dw[j][e];
      out[e] = 0.0f;
#pragma unroll
      for (int j = 0; j < K; ++j) out[e] = fmaf(w[j][e], dc[j][e], out[e]);
    }
    const int64_t s = t - (K - 1);  // the token whose gradient is complete
    if constexpr (kInside) {
      store_v(dx + s * P.D, out);
      return;
    }
    if (s < r.t0 && (s >= 0 || r.t0 > 0)) return;
    const int64_t m = s - (r.length - (K - 1));  // its place in the state behind the sequence
    if (P.dlast && m >= 0 && m < K - 1) {
      float g[V];
      load_v(static_cast<const T*>(P.dlast) + (r.b * (K - 1) + m) * P.D + r.c, g);
#pragma unroll
      for (int e = 0; e < V; ++e) out[e] += g[e];
    }
    if (s >= 0)
      store_v(dx + s * P.D, out);
    else if (P.dstate)
      store_v(static_cast<T*>(P.dstate) + (r.b * (K - 1) + K - 1 + s) * P.D + r.c, out);
  };
  auto load = [&](int64_t t, Raw<T, V>& in_x, Raw<T, V>& in_g) {
    if (end <= r.t0) return;  // (nothing of the run exists)
    t = t < end ? t : end - 1;
    load_raw<true>(x + t * P.ld_x, V, in_x);
    load_raw<true>(dy + t * P.ld_dy, V, in_g);
  };
  constexpr std::false_type kAny{};
  constexpr std::true_type kInside{};
  int64_t t = r.t0;
  Raw<T, V> one_x{}, one_g{};
  for (; t < stop && t < r.t0 + K - 1; ++t) {
    load(t, one_x, one_g);
    token(kAny, t, one_x, one_g);
  }
  const int64_t inner = end < r.t1 ? end : r.t1;
  if (t + kAhead <= inner) {
    Raw<T, V> nx[kAhead], ng[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) load(t + a, nx[a], ng[a]);
    for (; t + kAhead <= inner; t += kAhead) {
      Raw<T, V> ix[kAhead], ig[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        ix[a] = nx[a];
        ig[a] = ng[a];
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) load(t + kAhead + a, nx[a], ng[a]);
#pragma unroll
      for (int a = 0; a < kAhead; ++a) token(kInside, t + a, ix[a], ig[a]);
    }
  }
  for (; t < stop; ++t) {
    load(t, one_x, one_g);
    token(kAny, t, one_x, one_g);
  }
  float* to = P.parts + r.index * (K + 1) * P.D + r.c;
#pragma unroll
  for (int j = 0; j < K; ++j) store_v(to + j * P.D, dw[j]);
  store_v(to + K * P.D, dbias);
}

__global__ __launch_bounds__(1024) void conv_sums_kernel(const ConvRequest P) {
  column_sums(P.parts, P.B * P.runs, int64_t(P.K + 1) * P.D, [&](int64_t c, float sum) {
    const int64_t j = c / P.D, d = c % P.D;
    if (j < P.K)
      P.dw[d * P.K + j] = sum;
    else if (P.dbias)
      P.dbias[d] = sum;
  });
}

// One token: the state moves on by one input.  A thread owns its channels of one
// stream, state included, so the state may be updated in place.
template <typename T, int K, int V>
__global__ __launch_bounds__(256) void conv_step_kernel(const ConvRequest P) {
  const int64_t nvec = P.D / V;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= P.B * nvec) return;
  const int64_t b = i / nvec, c = i % nvec * V;
  float w[K][V], bias[V], win[K][V], out[V];
#pragma unroll
  for (int j = 0; j + 1 < K; ++j) input_at<T, K>(P, b, j + 1 - K, c, win[j]);
  load_v(static_cast<const T*>(P.x) + b * P.ld_x + c, win[K - 1]);
  load_taps<K>(P, c, w, bias);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float a = bias[e];
#pragma unroll
    for (int j = 0; j < K; ++j) a = fmaf(w[j][e], win[j][e], a);
    out[e] = P.silu ? a * logistic_f(a) : a;
  }
  store_v(static_cast<T*>(P.y) + b * P.D + c, out);
#pragma unroll
  for (int j = 1; j < K; ++j) store_v(static_cast<T*>(P.last) + (b * (K - 1) + j - 1) * P.D + c, win[j]);
}

// Calls f with the number of taps as a constant.
template <typename F>
void by_taps(int K, F f) {
  switch (K) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 5: return f(std::integral_constant<int, 5>{});
    case 6: return f(std::integral_constant<int, 6>{});
    case 7: return f(std::integral_constant<int, 7>{});
    default: return f(std::integral_constant<int, 8>{});
  }
}
// Calls f with the element type and a thread's channels: 16 bytes of them, or one
// where `whole` rows have fewer (the step: where they do not divide a row).
template <typename F>
void by_type(sr_dtype dtype, bool whole, F f) {
  if (dtype == SR_BF16) {
    if (whole)
      f(uint16_t{}, std::integral_constant<int, 8>{});
    else
      f(uint16_t{}, std::integral_constant<int, 1>{});
  } else {
    if (whole)
      f(float{}, std::integral_constant<int, 4>{});
    else
      f(float{}, std::integral_constant<int, 1>{});
  }
}

// A thread's channels: 16 bytes, in the backward pass (whose filter, windows and sums
// are all in registers) four: the call of 8 x 2048 x 1024 in bf16 31.3 us, with eight of them 33.6.
int64_t vector_of(sr_dtype dtype, bool backward) { return dtype == SR_BF16 && !backward ? 8 : 4; }

sr_status launched(const char* what) {
  const hipError_t err = hipGetLastError();
  return err == hipSuccess ? SR_OK : fail(SR_ERR_HIP, "%s: %s", what, hipGetErrorString(err));
}

}  // namespace

// Runs of tokens, 4 to 64 (the K - 1 inputs in front of a run are read again, in the
// backward pass the K - 1 behind it too): as long as two waves per SIMD are left, in the
// backward pass one.  Measured in us, bf16, runs of 4 / 8 / 16 / 32 / 64: 1 x 512 x 2048 4.4 / 5.3 / 7.0 / 11 / 18;
// 1 x 8192 x 2048 18.6 / 15.9 / 14.0 / 14.6 / 20.1; 8 x 4096 x 2048 58 / 51 / 46 / 46 / 45; backward
// 2 x 2048 x 512 18.5 / 14.6 / 14.4 / 17.2 / 25.4; 1 x 8192 x 2048 66 / 45 / 34 / 31 / 31.
ConvPlan conv_plan(int64_t B, int64_t T, int64_t D, sr_dtype dtype, bool backward) {
  const int64_t v = vector_of(dtype, backward), nvec = D >= v ? (D + v - 1) / v : D;
  const int64_t least = backward ? 65536 : 131072;  // threads
  ConvPlan plan{4, 0};
  while (plan.run_len < 64 && B * nvec * ((T + 2 * plan.run_len - 1) / (2 * plan.run_len)) >= least) plan.run_len *= 2;
  plan.runs = T > 0 ? (T + plan.run_len - 1) / plan.run_len : 1;  // (without tokens the states still pass)
  return plan;
}

int64_t conv_threads(const ConvRequest& P) {
  const int64_t v = vector_of(P.dtype, false), nvec = P.D >= v ? (P.D + v - 1) / v : P.D;
  return nvec * (P.B * P.runs + (P.last ? P.B * (P.K - 1) : 0));
}
int64_t conv_backward_threads(const ConvRequest& P) {
  const int64_t v = vector_of(P.dtype, true), nvec = P.D >= v ? (P.D + v - 1) / v : P.D;
  return nvec * P.B * P.runs;
}
int64_t conv_step_threads(const ConvRequest& P) {
  const int64_t v = vector_of(P.dtype, false);
  return P.B * (P.D % v == 0 ? P.D / v : P.D);
}

sr_status launch_conv(const ConvRequest& P) {
  const int64_t v = vector_of(P.dtype, false), n = conv_threads(P);
  if (n == 0) return SR_OK;
  by_type(P.dtype, P.D >= v, [&](auto t, auto width) {
    by_taps(P.K, [&](auto taps) {
      hipLaunchKernelGGL((conv_kernel<decltype(t), decltype(taps)::value, decltype(width)::value>),
                         dim3(uint32_t((n + 255) / 256)), dim3(256), 0, P.stream, P);
    });
  });
  return launched("convolution");
}

sr_status launch_conv_backward(const ConvRequest& P) {
  const int64_t v = vector_of(P.dtype, true), n = conv_backward_threads(P);
  by_type(P.dtype, P.D >= v, [&](auto t, auto width) {
    by_taps(P.K, [&](auto taps) {
      if (n > 0)
        hipLaunchKernelGGL((conv_backward_kernel<decltype(t), decltype(taps)::value, decltype(width)::value == 8 ? 4 : decltype(width)::value>),
                           dim3(uint32_t((n + 255) / 256)), dim3(256), 0, P.stream, P);
    });
  });
  sr_status st = launched("convolution backward");
  if (st != SR_OK) return st;
  hipLaunchKernelGGL(conv_sums_kernel, dim3(uint32_t(((P.K + 1) * P.D + 63) / 64)), dim3(1024), 0, P.stream, P);
  return launched("convolution gradient sums");
}

sr_status launch_conv_step(const ConvRequest& P) {
  const int64_t n = conv_step_threads(P);
  by_type(P.dtype, P.D % vector_of(P.dtype, false) == 0, [&](auto t, auto width) {
    by_taps(P.K, [&](auto taps) {
      hipLaunchKernelGGL((conv_step_kernel<decltype(t), decltype(taps)::value, decltype(width)::value>),
                         dim3(uint32_t((n + 255) / 256)), dim3(256), 0, P.stream, P);
    });
  });
  return launched("convolution step");
}

}  // namespace sr
