// 8-bit integer product with a scale per row of either operand, and the
// single-token minGRU step on it:
//
//     c[m, n] = (sum_k a[m, k] b[n, k]) (s_m t_n)
//
// The sum is exact in 32-bit integers (|a|, |b| <= 127 and K <= kMaxI8Depth
// keep it below 2^31), so neither the order of the sum nor the tiling
// changes a result; it is rounded once to fp32, multiplied by the product of
// the scales, and rounded once more if the output is bf16.
//
// In every kernel the weights are the left operand of the matrix
// instruction, so that a lane ends with four consecutive output columns of
// one row: 16-byte stores, and in the step four channels whose states are one
// 16-byte load and store.  Operands reach LDS by direct loads through buffer
// descriptors that end with the tile's last row: rows past the end read as
// zeros, with no test in the kernel.
//
// i8_narrow_kernel  tiles of up to 64 x 64, the depth split over the waves:
//                   products that 128 x 128 tiles would leave CUs without
//                   (a step over up to a few hundred streams).
// i8_token_kernel   the same for up to four rows that are not quantised yet.
// i8_large_kernel   tiles of 128 x 128 and 256 x 256, persistent.

#include "internal.hpp"
#include "quant.hpp"
#include "step_gate.hpp"

namespace sr {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
using rsrc_t = __amdgpu_buffer_rsrc_t;

enum Out { kF32 = 0, kBF16 = 1, kStep = 2, kStepDecay = 3 };
constexpr bool is_step(int out) { return out >= kStep; }

constexpr int kDepth = 128;             // bytes of K per stage: whole lines
constexpr int kRsrcWord3 = 0x00020000;  // raw buffer, gfx9 format
constexpr int kNonTemporal = 2;         // cache policy of a store
constexpr int kCus = 256;

struct I8Params {
  int64_t M, N, K;  // N: output columns (step: 2 D_h); K: stored width, a multiple of kI8Align
  const int8_t* A;
  int64_t lda;
  const float* a_scale;  // [M]
  const int8_t* B;
  int64_t ldb;
  const float* b_scale;  // [N]
  void* C;               // [M, N], rows of ldc elements
  int64_t ldc;
  bool lines;            // rows of C start at multiples of 128 bytes
  uint32_t tiles_m, tiles_n, n_tiles;
  // tokens: the rows of X are quantised by the kernel, A and a_scale are unused
  const void* X;  // [M, Kx], contiguous
  int Kx;
  // step: k and p are columns d and D_h + d
  int64_t D_h;
  const float* h_prev;
  float* h_next;
  const float* rate;
  const float* gap;
  int log1p_gap;
  uint32_t* saturated;
};

// A descriptor over `bytes` from base; reads past its end return zeros.
__device__ __forceinline__ rsrc_t buffer(const void* base, int64_t bytes) {
  const int64_t n = bytes < 0 ? 0 : (bytes > int64_t(0xFFFFFFFF) ? int64_t(0xFFFFFFFF) : bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, int(uint32_t(n)), kRsrcWord3);
}
__device__ __forceinline__ f32x4 load4(rsrc_t r, int byte) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, byte, 0, 0));
}
// 16 bytes per lane straight to LDS, lane l's at lds + 16 l.
__device__ __forceinline__ void load_lds(rsrc_t r, int8_t* lds, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, soff, 0, 0);
}
// Waits until at most N of this wave's loads are outstanding and all its LDS
// reads have returned.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// (Products here and in decayed() are rounded on their own, never joined with
// a later sum: a row's results do not depend on the kernel that makes them.)
__device__ __forceinline__ float scaled(int acc, float s, float t) {
#pragma clang fp contract(off)
  return float(acc) * (s * t);
}

// The states h entering the step at four channels whose decay rates are rate
// (zero past the last), of a row with this time gap: with time decay each is
// scaled by exp(-min(rate gap, 1e4)).
__device__ __forceinline__ f32x4 decayed(const I8Params& P, float gap, f32x4 rate, f32x4 h) {
#pragma clang fp contract(off)
  constexpr float kClamp = 1.0e4f, kLog2e = 1.4426950408889634f;
  if (P.log1p_gap) gap = log1pf(gap);
  bool saturated = false;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float e = rate[r] * gap;
    saturated |= e > kClamp;
    h[r] *= __builtin_amdgcn_exp2f(fminf(e, kClamp) * -kLog2e);
  }
  if (saturated && P.saturated != nullptr)
    __hip_atomic_fetch_or(P.saturated, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return h;
}
// The same of row m < M, channels from d.
__device__ __forceinline__ f32x4 decayed(const I8Params& P, int64_t m, int64_t d, f32x4 h) {
  return decayed(P, P.gap[m], load4(buffer(P.rate, P.D_h * 4), int(d) * 4), h);
}

// Four consecutive results of row m from column n (step: channel n).
template <int OUT>
__device__ __forceinline__ void store4(const I8Params& P, int64_t m, int64_t n, f32x4 v) {
  const int64_t end = is_step(OUT) ? P.D_h : P.N;
  if (m >= P.M || n >= end) return;
  if constexpr (OUT == kBF16) {
    uint16_t* dst = static_cast<uint16_t*>(P.C) + m * P.ldc + n;
    if (n + 4 <= end) {
      u32x2 w;
      w.x = bf16_pair(v[0], v[1]);
      w.y = bf16_pair(v[2], v[3]);
      __builtin_memcpy(__builtin_assume_aligned(dst, 2), &w, 8);  // one store at any even address
    } else {
#pragma unroll 1
      for (int j = 0; j < 4 && n + j < end; ++j) {
        dst[j] = uint16_t(bf16_pair(v[0], v[0]));
        v = f32x4{v[1], v[2], v[3], v[3]};
      }
    }
  } else {
    float* dst = is_step(OUT) ? P.h_next + m * P.D_h + n : static_cast<float*>(P.C) + m * P.ldc + n;
    if (n + 4 <= end) {
      __builtin_memcpy(__builtin_assume_aligned(dst, 4), &v, 16);
    } else {
#pragma unroll 1
      for (int j = 0; j < 4 && n + j < end; ++j) {
        dst[j] = v[0];
        v = f32x4{v[1], v[2], v[3], v[3]};
      }
    }
  }
}

// Consecutive workgroups go to the XCDs round-robin; renumbered, each XCD has
// a contiguous range of tiles, which share operands in its L2.
__device__ __forceinline__ uint32_t xcd_tile(uint32_t n) {
  const uint32_t per = n / 8;
  return blockIdx.x < per * 8 ? (blockIdx.x % 8) * per + blockIdx.x / 8 : blockIdx.x;
}

// -------------------------------------------------- product of few rows

// A workgroup of four waves owns 16 MT rows x 16 NT columns (step: half as
// many channels, a block of k columns and one of p in turn) and splits the
// depth over its waves: wave w multiplies the whole tile over every fourth
// 128-byte line.  Each wave brings its lines to its own part of LDS and waits
// on its own loads only; two lines per wave, the next one loading while one
// is multiplied.  Each byte is read once per workgroup, and nobody meets at a
// barrier until the waves' sums do in LDS (integers: their order does not
// matter).  256 x 2048 x 4096 takes 7.2 us, 600 TOP/s: 256 tiles of 64 x 64 move
// 64 MB from L2, at 22 TB/s.
// v_mfma_i32_16x16x64_i8: lane l supplies 16 consecutive bytes of row l % 16
// from 16 (l / 16); accumulator r of lane l is D[4 (l / 16) + r][l % 16].
constexpr int kSplitWaves = 4;

template <int OUT, int MT, int NT>
struct NarrowTile {
  static constexpr int kRows = 16 * (MT + NT);
  static constexpr int kLoads = kRows / 8;
  static constexpr int kLineBytes = kRows * kDepth;
  static constexpr int kPair = is_step(OUT) ? 2 : 1;
  static constexpr int kParts = MT * NT / kPair;
  static constexpr int kMine = (kParts + kSplitWaves - 1) / kSplitWaves;
  static_assert(!is_step(OUT) || NT % 2 == 0, "k and p blocks alternate");

  const I8Params& P;
  int lane, wave;
  rsrc_t ra, rb;
  int va[2], vb[2];  // this lane's offset in eight rows of A or B, for even and odd eights
  int roff[2];
  i32x4 acc[MT][NT];

  // An instruction brings eight rows' 128 bytes; place c ^ (r / 2 % 8) of row
  // r holds its 16-byte chunk c, which spreads an operand read of 16 rows over
  // all 64 banks.
  __device__ __forceinline__ void aim(int64_t m0, int64_t n0) {
    ra = buffer(P.A + m0 * P.lda, (P.M - m0 - 1) * P.lda + P.K);
    rb = buffer(P.B + n0 * P.ldb, (P.N - n0 - 1) * P.ldb + P.K);
    const int lrow = lane >> 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int chunk = ((lane & 7) ^ (h * 4 + (lrow >> 1))) * 16;
      va[h] = lrow * int(P.lda) + chunk;
      vb[h] = lrow * int(P.ldb) + chunk;
      roff[h] = (lane & 15) * kDepth + (((h * 4 + (lane >> 4)) ^ ((lane >> 1) & 7)) << 4);
    }
  }
  __device__ __forceinline__ void load(int8_t* __restrict__ dst, int i) {
    const int k = (i * kSplitWaves + wave) * kDepth;
#pragma unroll
    for (int q = 0; q < 2 * MT; ++q) load_lds(ra, dst + q * 1024, va[q & 1], q * 8 * int(P.lda) + k);
#pragma unroll
    for (int q = 0; q < 2 * NT; ++q) {
      const int block = q / 2;
      const uint32_t row = uint32_t(block / kPair * 16 + (q & 1) * 8);
      uint32_t soff = row * uint32_t(P.ldb) + uint32_t(k);
      if (is_step(OUT) && block % 2) soff += uint32_t(P.D_h) * uint32_t(P.ldb);
      load_lds(rb, dst + (2 * MT + q) * 1024, vb[q & 1], int(soff));
    }
  }
  // Multiplies line i (if it is one), and brings line i + 2 to its place.
  __device__ __forceinline__ void line(int8_t* __restrict__ cur, int i, int n) {
    i32x4 a[2][MT], b[2][NT];
    if (i >= 0) {
      if (i + 1 < n)
        wait_loads<kLoads>();
      else
        wait_loads<0>();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int m = 0; m < MT; ++m) a[h][m] = *reinterpret_cast<const i32x4*>(cur + m * 16 * kDepth + roff[h]);
#pragma unroll
        for (int j = 0; j < NT; ++j)
          b[h][j] = *reinterpret_cast<const i32x4*>(cur + (MT + j) * 16 * kDepth + roff[h]);
      }
    }
    if (i + 2 < n) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the reads have left the buffer
      load(cur, i + 2);
    }
    if (i >= 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            acc[m][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[h][j], a[h][m], acc[m][j], 0, 0, 0);
    }
  }
  __device__ __forceinline__ void run(int8_t* __restrict__ p0, int8_t* __restrict__ p1, int n) {
    for (int i = -2; i < n; i += 2) {
      line(p0, i, n);
      if (i + 1 < n) line(p1, i + 1, n);
    }
  }
};

template <int OUT, int MT, int NT>
__global__ __launch_bounds__(64 * kSplitWaves) void i8_narrow_kernel(const I8Params P) {
  using T = NarrowTile<OUT, MT, NT>;
  constexpr int W = kSplitWaves, kPair = T::kPair;
  constexpr int kStaging = W * 2 * T::kLineBytes, kSums = W * MT * NT * 1024;
  __shared__ __align__(1024) int8_t smem[kStaging > kSums ? kStaging : kSums];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Row tiles fast: those of a column tile share its weights.
  const uint32_t tile = xcd_tile(gridDim.x);
  const int64_t m0 = int64_t(tile % P.tiles_m) * (16 * MT);
  const int64_t n0 = int64_t(tile / P.tiles_m) * (16 * NT / kPair);
  T t{P, lane, wave};
  t.aim(m0, n0);

  // Scales and states of the parts this wave finishes, first in the queue.
  f32x4 sb[T::kMine][kPair], hp[T::kMine];
  float sa[T::kMine];
  int pm[T::kMine], pn[T::kMine];  // this lane's row and first column within the tile
  const rsrc_t rs = buffer(P.a_scale + m0, (P.M - m0) * 4);
  const rsrc_t rt = buffer(P.b_scale + n0, (P.N - n0) * 4);
  const rsrc_t rh = buffer(is_step(OUT) && P.h_prev != nullptr ? P.h_prev + m0 * P.D_h + n0 : nullptr,
                           is_step(OUT) && P.h_prev != nullptr ? ((P.M - m0) * P.D_h - n0) * 4 : 0);
#pragma unroll
  for (int q = 0; q < T::kMine; ++q) {
    const int block = (q * W + wave) * kPair;
    pm[q] = block / NT * 16 + (lane & 15);
    pn[q] = block % NT / kPair * 16 + 4 * (lane >> 4);
    sa[q] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, pm[q] * 4, 0, 0));
#pragma unroll
    for (int h = 0; h < kPair; ++h)
      sb[q][h] = load4(rt, (pn[q] + h * int(P.D_h)) * 4);
    if constexpr (is_step(OUT)) hp[q] = load4(rh, (pm[q] * int(P.D_h) + pn[q]) * 4);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) t.acc[m][j] = i32x4{};
  int8_t* mine = smem + wave * 2 * T::kLineBytes;
  t.run(mine, mine + T::kLineBytes, (int(P.K / kDepth) - wave + W - 1) / W);

  __syncthreads();  // every wave is done with its lines: the sums take their place
  i32x4* sums = reinterpret_cast<i32x4*>(smem);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) sums[((m * NT + j) * W + wave) * 64 + lane] = t.acc[m][j];
  __syncthreads();
#pragma unroll
  for (int q = 0; q < T::kMine; ++q) {
    const int part = q * W + wave;
    if (part >= T::kParts) break;
    i32x4 sum[kPair];
#pragma unroll
    for (int h = 0; h < kPair; ++h) {
      const i32x4* from = sums + (part * kPair + h) * W * 64 + lane;
      sum[h] = from[0];
#pragma unroll
      for (int w = 1; w < W; ++w) sum[h] += from[w * 64];
    }
    f32x4 v;
    if constexpr (is_step(OUT)) {
      if constexpr (OUT == kStepDecay)
        if (m0 + pm[q] < P.M) hp[q] = decayed(P, m0 + pm[q], n0 + pn[q], hp[q]);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        v[r] = step_value(scaled(sum[0][r], sa[q], sb[q][0][r]), scaled(sum[1][r], sa[q], sb[q][1][r]), hp[q][r]);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = scaled(sum[0][r], sa[q], sb[q][0][r]);
    }
    store4<OUT>(P, m0 + pm[q], n0 + pn[q], v);
  }
}

// ------------------------------------------------------------------ tokens

// Up to four rows (single tokens of a few streams) against 16 columns (step:
// eight channels) per workgroup, where a launch of its own for the codes would
// cost as much as the product.  Every weight is used by one wave only, so each
// wave loads its share, every fourth 128-byte line, straight to registers, all
// of it before anything else is done; meanwhile the workgroup quantises the
// rows into LDS.  The codes are those of the quantisation kernels.  Bound by
// the latency of the launch and of the weights, from D = 4096 by their bytes.
// Measured (us, a step's state alone, D x 2 D weights from four alternating
// buffers, one launch after the other):
//   rows x D                    1 x 512  4 x 512  1 x 2048  4 x 2048  1 x 4096  4 x 4096
//   codes, then their product     4.7      5.0      6.2       6.5      10.0      10.4
//   this kernel                   3.2      3.1      4.6       5.1       8.3       9.8
//   with 32 columns               3.4      3.3      6.2       6.8       8.6       9.7
constexpr int kMaxTokens = 4;
constexpr int kMaxTokenDepth = 4096;

// DEPTH: the longest row.
template <int OUT, typename TX, int DEPTH>
__global__ __launch_bounds__(64 * kSplitWaves) void i8_token_kernel(const I8Params P) {
  using C = Chunk<TX>;
  constexpr int W = kSplitWaves, R = kMaxTokens, kLines = DEPTH / kDepth / W;
  constexpr int kChunks = DEPTH / C::kSize / 64;  // of a row, for one wave's lanes
  constexpr int kCols = is_step(OUT) ? 8 : 16;
  constexpr int kPair = is_step(OUT) ? 2 : 1;
  __shared__ __align__(16) int8_t s_codes[R * DEPTH];
  __shared__ i32x4 s_sums[W * 64];
  __shared__ uint32_t s_top[W];
  __shared__ float s_scale[W];
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = int64_t(xcd_tile(gridDim.x)) * kCols;

  // A row is quantised by four waves (one row), by two (two) or by one.  The
  // lane's chunks of it, zeros past its end; loads end in order, so these come
  // first.
  const int wpr_log = P.M == 1 ? 2 : P.M == 2 ? 1 : 0;
  const int row = wave >> wpr_log, c0 = ((wave & ((1 << wpr_log) - 1)) << 6) + lane;
  const bool quantises = row < P.M;
  const rsrc_t rx = buffer(static_cast<const TX*>(P.X) + int64_t(row) * P.Kx,
                           quantises ? P.Kx * int(sizeof(TX)) : 0);
  u32x4 x[kChunks];
#pragma unroll
  for (int j = 0; j < kChunks; ++j)
    x[j] = __builtin_amdgcn_raw_buffer_load_b128(rx, (c0 + (j << (6 + wpr_log))) * 16, 0, 0);
  __builtin_amdgcn_sched_barrier(0);

  // This wave's weights: line i * W + wave; zeros for lines past the last.
  // Step: eight rows of k, then the eight of p.
  u32x4 b[kLines][2];
  const int brow = is_step(OUT) && (lane & 8) ? int(P.D_h) + (lane & 7) : (lane & 15);
  const int boff = int(uint32_t(brow) * uint32_t(P.ldb)) + g * 16;
  const int64_t b_bytes = (P.N - n0 - 1) * P.ldb + P.K;
#pragma unroll
  for (int i = 0; i < kLines; ++i) {
    const int k = (i * W + wave) * kDepth;
    const rsrc_t rb = buffer(P.B + n0 * P.ldb, k < P.K ? b_bytes : 0);
#pragma unroll
    for (int h = 0; h < 2; ++h) b[i][h] = __builtin_amdgcn_raw_buffer_load_b128(rb, boff, k + h * 64, 0);
  }
  // Scales and states of the results this lane finishes: row m, four columns from n.
  const int m = lane & 15;
  const int64_t n = n0 + (is_step(OUT) ? g % 2 : g) * 4;
  f32x4 sb[kPair], hp{};
  const rsrc_t rt = buffer(P.b_scale + n0, (P.N - n0) * 4);
#pragma unroll
  for (int h = 0; h < kPair; ++h) sb[h] = load4(rt, int(n - n0 + h * P.D_h) * 4);
  if (is_step(OUT) && P.h_prev != nullptr)
    hp = load4(buffer(P.h_prev + n0, (P.M * P.D_h - n0) * 4), int(m * P.D_h + n - n0) * 4);
  __builtin_amdgcn_sched_barrier(0);

  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const uint32_t t = C::top(x[j]);
    top = top > t ? top : t;
  }
  top = wave_max(top);
  if (lane == 0) s_top[wave] = top;
  __syncthreads();
  if (quantises) {
    for (int w = 1; w < 1 << wpr_log; ++w) {
      const uint32_t t = s_top[wave ^ w];
      top = top > t ? top : t;
    }
    const float s = row_scale(top);
    if (lane == 0) s_scale[row] = s;
    const bool plain = divides_plainly(s);
    const float rs = plain ? __fdiv_rn(1.0f, s) : 0.0f;
    // 128 bytes of a line a row, row r's 16-byte chunk c at c ^ 4 (r / 2), so
    // that the halves of four rows lie in different banks.
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int k = (c0 + (j << (6 + wpr_log))) * C::kSize;
      if (((j * 64) << wpr_log) * C::kSize < P.K) {
        uint32_t c[C::kSize / 4];
        C::codes(x[j], s, rs, plain, c);
        if (k < P.K) {
          int8_t* at = s_codes + (k / kDepth * R + row) * kDepth + (((k % kDepth / 16) ^ (row / 2 * 4)) << 4) + k % 16;
#pragma unroll
          for (int d = 0; d < C::kSize / 4; ++d) reinterpret_cast<uint32_t*>(at)[d] = c[d];
        }
      }
    }
  }
  __syncthreads();

  // The tile's 16 rows are the four over and over; only the first M are stored.
  i32x4 acc{};
  const int arow = lane % R;
  const float s_row = s_scale[arow];
#pragma unroll
  for (int i = 0; i < kLines; ++i) {
    const int line = i * W + wave;
    if (line * kDepth < P.K) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const i32x4 a = *reinterpret_cast<const i32x4*>(s_codes + (line * R + arow) * kDepth +
                                                        (((h * 4 + g) ^ (arow / 2 * 4)) << 4));
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(i32x4(b[i][h]), a, acc, 0, 0, 0);
      }
    }
  }
  s_sums[threadIdx.x] = acc;
  __syncthreads();
  if (wave > 0 || m >= P.M || g >= 4 / kPair) return;
  i32x4 sum[kPair];  // step: k's, and p's from the lanes 32 on
#pragma unroll
  for (int h = 0; h < kPair; ++h) {
    const i32x4* from = s_sums + lane + h * 32;
    sum[h] = from[0];
#pragma unroll
    for (int w = 1; w < W; ++w) sum[h] += from[w * 64];
  }
  f32x4 v;
  if constexpr (is_step(OUT)) {
    if constexpr (OUT == kStepDecay) hp = decayed(P, m, n, hp);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      v[r] = step_value(scaled(sum[0][r], s_row, sb[0][r]), scaled(sum[1][r], s_row, sb[1][r]), hp[r]);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = scaled(sum[0][r], s_row, sb[0][r]);
  }
  store4<OUT>(P, m, n, v);
}

// ------------------------------------------------------------- large product

// Tiles of 64 MB x 64 NB results, four waves of 32 MB x 32 NB each, as 32 x
// 32 x 32 products; persistent workgroups.  Two LDS stages of 128 bytes of
// depth; the stage two ahead is loaded into the buffer that the current one
// leaves, across tiles too, so that a tile's results are stored under the
// next one's first loads.  With MB = NB = 4 a lane holds 256 sums, a CU one
// workgroup, and an operand byte that a wave reads from LDS is used 128 times.
// 131072 x 2048 x 4096 with bf16 results takes 1052 to 1077 us, 2.0 to 2.1 POP/s:
// the matrix cores are busy half of the cycles, at 1.75 GHz (8192^3: 63% at 1.66
// GHz; the clock falls as they are busier).
// v_mfma_i32_32x32x32_i8: lane l supplies 16 consecutive bytes of row l % 32
// from 16 (l / 32); accumulator r of lane l is D[8 (r / 4) + 4 (l / 32) + r % 4][l % 32].
template <int MB_, int NB_>
struct LargeShape {
  static constexpr int MB = MB_, NB = NB_, R = 32, KS = 4, kWaves = 4;
  static constexpr int kM = 64 * MB, kN = 64 * NB;
  static constexpr int kLoadsA = kM / 8 / kWaves, kLoadsB = kN / 8 / kWaves;  // per wave and stage
  static constexpr int kLoads = kLoadsA + kLoadsB;
  static constexpr int kStageBytes = (kM + kN) * kDepth;
  static constexpr int kOutRow = 64 * NB;        // bytes of a row of results in LDS
  static constexpr int kOutBytes = R * kOutRow;  // per wave
  static constexpr int kLds = 2 * kStageBytes + kWaves * kOutBytes;
  static constexpr int kPerCu = 160 * 1024 / kLds;
  static_assert(kWaves == 4, "the order of the loads");
};

template <int OUT, class S>
struct LargeTile {
  static constexpr int MB = S::MB, NB = S::NB, R = S::R;
  static constexpr int kSpan = is_step(OUT) ? S::kN / 2 : S::kN;  // columns (channels) of a tile
  const I8Params& P;
  int lane, wave, wm, wn;
  rsrc_t ra, rb;
  int va, vb;  // this lane's offset in eight rows of A or B
  int roff[S::KS];
  i32x4 fa[2][MB], fb[2][NB];
  i32x16 acc[MB][NB];

  // Tiles in groups of kGroupM tile rows, column by column within a group: the
  // 32 tiles that run on an XCD at a time share 8 row and 4 column tiles.
  // Measured (131072 x 2048 x 4096, bf16 results): groups of 2, 4, 8, 16 rows
  // 1185, 1094, 1062, 1069 us.
  __device__ __forceinline__ void origin(uint32_t t, int64_t& m0, int64_t& n0) const {
    constexpr uint32_t kGroupM = 8;
    const uint32_t per_group = kGroupM * P.tiles_n;
    const uint32_t g = t / per_group, in = t % per_group;
    const uint32_t left = P.tiles_m - g * kGroupM;
    const uint32_t rows = left < kGroupM ? left : kGroupM;
    m0 = int64_t(g * kGroupM + in % rows) * S::kM;
    n0 = int64_t(in / rows) * kSpan;
  }
  __device__ __forceinline__ void aim(uint32_t t) {
    int64_t m0, n0;
    origin(t, m0, n0);
    ra = buffer(P.A + m0 * P.lda, (P.M - m0 - 1) * P.lda + P.K);
    rb = buffer(P.B + n0 * P.ldb, (P.N - n0 - 1) * P.ldb + P.K);
  }
  // Swizzled as in NarrowTile; wave w takes the eights w, w + 4, ... of the rows.
  __device__ __forceinline__ void lanes() {
    const int lrow = lane >> 3, chunk = ((lane & 7) ^ ((wave & 1) * 4 + (lrow >> 1))) * 16;
    va = lrow * int(P.lda) + chunk;
    vb = lrow * int(P.ldb) + chunk;
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks)
      roff[ks] = (lane % R) * kDepth + (((ks * 2 + lane / R) ^ ((lane >> 1) & 7)) << 4);
  }
  // Stage kt of the tile aimed at.  A single-stage product has a second one
  // past its end, of zeros (one without depth has two): no descriptor reaches that far.
  __device__ __forceinline__ void load_stage(int8_t* __restrict__ dst, uint32_t kt) {
    const bool past = int64_t(kt) * kDepth >= P.K;
    const rsrc_t a = past ? buffer(nullptr, 0) : ra, b = past ? buffer(nullptr, 0) : rb;
    uint32_t soff = uint32_t(wave * 8) * uint32_t(P.lda) + kt * kDepth;
#pragma unroll
    for (int q = 0; q < S::kLoadsA; ++q) {
      load_lds(a, dst + (q * S::kWaves + wave) * 1024, va, int(soff));
      soff += uint32_t(8 * S::kWaves) * uint32_t(P.lda);
    }
    // Step: a block of 32 columns is k of 16 channels, then their p.
    soff = (is_step(OUT) ? uint32_t(wave % 2 * 8) + uint32_t(wave / 2) * uint32_t(P.D_h) : uint32_t(wave * 8)) *
               uint32_t(P.ldb) + kt * kDepth;
#pragma unroll
    for (int q = 0; q < S::kLoadsB; ++q) {
      load_lds(b, dst + S::kM * kDepth + (q * S::kWaves + wave) * 1024, vb, int(soff));
      soff += uint32_t(is_step(OUT) ? 16 : 32) * uint32_t(P.ldb);
    }
  }
  __device__ __forceinline__ void read(int set, const int8_t* __restrict__ src, int ks) {
    const int8_t* a = src + wm * (MB * R * kDepth) + roff[ks];
    const int8_t* b = src + (S::kM + wn * NB * R) * kDepth + roff[ks];
#pragma unroll
    for (int i = 0; i < MB; ++i) fa[set][i] = *reinterpret_cast<const i32x4*>(a + i * R * kDepth);
#pragma unroll
    for (int j = 0; j < NB; ++j) fb[set][j] = *reinterpret_cast<const i32x4*>(b + j * R * kDepth);
  }
  // One stage: its products, with the first operands of the next one read and
  // stage load_kt loaded into the buffer it leaves.
  __device__ __forceinline__ void stage(int8_t* __restrict__ cur, int8_t* __restrict__ nxt,
                                        uint32_t load_kt) {
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) {
      const int set = ks & 1;
      if (ks + 1 < S::KS) {
        read(set ^ 1, cur, ks + 1);
      } else {
        // The last of this stage is in registers and the next one has
        // landed: once every wave is here, the buffers change roles.
        wait_loads<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        read(set ^ 1, nxt, 0);
        load_stage(cur, load_kt);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[set][j], fa[set][i], acc[i][j], 0, 0, 0);
      if (ks + 1 < S::KS) {
        // Spread the operand reads over the products that hide them.
#pragma unroll
        for (int q = 0; q < MB + NB; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                    // an LDS read
          __builtin_amdgcn_sched_group_barrier(0x008, MB * NB / (MB + NB), 0);  // products
        }
      }
    }
  }
  // A tile's products and results; p0 holds stage kt of it, p1 the next one;
  // an even number of stages is left.
  __device__ __forceinline__ void run(int8_t* __restrict__ p0, int8_t* __restrict__ p1,
                                      int8_t* __restrict__ out, uint32_t n_kt, uint32_t kt,
                                      uint32_t tile, uint32_t next) {
    for (; kt + 2 < n_kt; kt += 2) {
      stage(p0, p1, kt + 2);
      stage(p1, p0, kt + 3);
    }
    aim(next);
    stage(p0, p1, 0);
    stage(p1, p0, 1);
    if constexpr (is_step(OUT)) {
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          States<1, 1> st;
          load_states(st, tile, i, j);
          update(out, st, i, j);
        }
    } else {
      store(out, tile);
    }
  }
  // What the states of a step come from, but the sums: h_prev, scales (and
  // decay) of MBP x NBP blocks of 32 rows x 16 channels from block (i, j) on, for
  // one row and four channels per lane and iteration, a row's by lanes side by
  // side.
  template <int MBP, int NBP>
  struct States {
    static constexpr int kPerRow = 4 * NBP, kRows = 64 / kPerRow, kIts = MBP * R / kRows;
    int64_t m, n;  // of this lane's first row and channel
    f32x4 h[kIts], tk, tp, rate;
    float s[kIts], gap[kIts];
  };
  template <int MBP, int NBP>
  __device__ __forceinline__ void load_states(States<MBP, NBP>& st, uint32_t tile, int i, int j) const {
    using St = States<MBP, NBP>;
    int64_t m0, n0;
    origin(tile, m0, n0);
    m0 += wm * (MB * R) + i * R;
    n0 += wn * (NB * R / 2) + j * 16;
    const int r = lane / St::kPerRow, c = lane % St::kPerRow * 4;
    st.m = m0 + r;
    st.n = n0 + c;
    const rsrc_t rs = buffer(P.a_scale + m0, (P.M - m0) * 4), rt = buffer(P.b_scale + n0, (P.N - n0) * 4);
    const rsrc_t rh = buffer(P.h_prev + m0 * P.D_h + n0, P.h_prev == nullptr ? 0 : ((P.M - m0) * P.D_h - n0) * 4);
    st.tk = load4(rt, c * 4);
    st.tp = load4(rt, (c + int(P.D_h)) * 4);
    if constexpr (OUT == kStepDecay) st.rate = load4(buffer(P.rate + n0, (P.D_h - n0) * 4), c * 4);
#pragma unroll
    for (int it = 0; it < St::kIts; ++it) {
      const int row = r + it * St::kRows;
      st.h[it] = load4(rh, int(uint32_t(row) * uint32_t(P.D_h) + uint32_t(c)) * 4);
      st.s[it] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, row * 4, 0, 0));
      if constexpr (OUT == kStepDecay)
        st.gap[it] = __uint_as_float(
            __builtin_amdgcn_raw_buffer_load_b32(buffer(P.gap + m0, (P.M - m0) * 4), row * 4, 0, 0));
    }
  }
  // The new states of those blocks.  The sums pass through LDS, a block's k and
  // p side by side in 128 bytes a row, so that the gates are one short loop and
  // a row's states are stored by lanes side by side: unrolled over the sums'
  // registers they were 16 KB of instructions (1024 x 2048: 24.3 -> 22.7 us with
  // its quantisation).  A gate is 24 instructions, four of them transcendental:
  // 2 us per tile of 128 x 128.  Place c ^ row % 8 of a row holds its 16-byte
  // chunk c.
  template <int MBP, int NBP>
  __device__ __forceinline__ void update(int8_t* __restrict__ out, States<MBP, NBP>& st, int i, int j) {
    using St = States<MBP, NBP>;
#pragma unroll
    for (int ii = 0; ii < MBP; ++ii)
#pragma unroll
      for (int jj = 0; jj < NBP; ++jj)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int row = lane % R, chunk = 2 * g + lane / R;
          const i32x16& a = acc[i + ii][j + jj];
          *reinterpret_cast<i32x4*>(out + ((ii * NBP + jj) * R + row) * 128 + ((chunk ^ (row & 7)) << 4)) =
              i32x4{a[4 * g], a[4 * g + 1], a[4 * g + 2], a[4 * g + 3]};
        }
    const int jj = lane % St::kPerRow / 4, chunk = lane % 4;
#pragma unroll 1
    for (int it = 0; it < St::kIts; ++it) {
      const int by = it * St::kRows, r = lane / St::kPerRow + by, row = r % R;
      const int8_t* from = out + ((r / R * NBP + jj) * R + row) * 128;
      const i32x4 k = *reinterpret_cast<const i32x4*>(from + ((chunk ^ (row & 7)) << 4));
      const i32x4 p = *reinterpret_cast<const i32x4*>(from + (((chunk + 4) ^ (row & 7)) << 4));
      f32x4 h = st.h[0], v;
      if constexpr (OUT == kStepDecay)
        if (st.m + by < P.M) h = decayed(P, st.gap[0], st.rate, h);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = step_value(scaled(k[e], st.s[0], st.tk[e]), scaled(p[e], st.s[0], st.tp[e]), h[e]);
      store4<OUT>(P, st.m + by, st.n, v);
#pragma unroll
      for (int q = 0; q + 1 < St::kIts; ++q) {
        st.h[q] = st.h[q + 1];
        st.s[q] = st.s[q + 1];
        if constexpr (OUT == kStepDecay) st.gap[q] = st.gap[q + 1];
      }
    }
  }

  // The wave's results, 32 rows x kOutRow bytes at a time through LDS, so that
  // neighbouring lanes store one row's bytes.  Place c ^ row % (chunks per
  // row) of a row holds its 16-byte chunk c.
  __device__ __forceinline__ void store(int8_t* __restrict__ out, uint32_t tile) {
    constexpr int kSize = OUT == kBF16 ? 2 : 4;
    constexpr int kChunks = S::kOutRow / 16;
    constexpr int kPassN = S::kOutRow / kSize / R;  // column blocks per pass
    constexpr int kPer = 16 / kSize;                // results per chunk
    constexpr int kRowsPer = 64 / kChunks;          // rows per store instruction
    int64_t m0, n0;
    origin(tile, m0, n0);
    m0 += wm * (MB * R);
    n0 += wn * (NB * R);
    const int rows = int(P.M - m0 < MB * R ? P.M - m0 : MB * R);  // may be negative: nothing here
    const int cols = int(P.N - n0 < NB * R ? P.N - n0 : NB * R);
    if (rows <= 0 || cols <= 0) return;
    // Scales past the end read as zero.
    const rsrc_t rs = buffer(P.a_scale + m0, rows * 4), rt = buffer(P.b_scale + n0, cols * 4);
    float s[MB];
    f32x4 t[NB][4];
#pragma unroll
    for (int i = 0; i < MB; ++i)
      s[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, (i * R + lane % R) * 4, 0, 0));
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        t[j][g] = load4(rt, (j * R + 8 * g + 4 * (lane / R)) * 4);
    const bool wide = P.ldc <= (int64_t(1) << 20);  // 32-bit offsets
    // The largest products' results leave the caches to the operands (131072 x
    // 512 x 1024 fp32: 164 -> 134 us); where lines are shared by two rows of
    // results, that would write them twice (20000 x 2048 x 1000: 55 -> 65 us).
    const bool stream = S::MB == 4 && P.lines;
    const int row = lane % R, swz = row % kChunks;
    const int tail = cols % kPer * kSize, tail_n = cols - cols % kPer;  // bytes past the last whole chunk, its end
    const int c = lane % kChunks, r0 = lane / kChunks;
    char* dst = static_cast<char*>(P.C) + (m0 * P.ldc + n0) * kSize;
    const rsrc_t rc = buffer(dst, int64_t(0xFFFFFFFF));
    const int row_bytes = int(P.ldc) * kSize;
    const int voff_c = r0 * row_bytes + c * 16;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
#pragma unroll
      for (int pass = 0; pass < NB / kPassN; ++pass) {
#pragma unroll
        for (int jj = 0; jj < kPassN; ++jj) {
          const int j = pass * kPassN + jj;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            f32x4 v;
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = scaled(acc[i][j][4 * g + r], s[i], t[j][g][r]);
            const int byte = (jj * R + 8 * g + 4 * (lane / R)) * kSize;
            int8_t* at = out + row * S::kOutRow + (((byte >> 4) ^ swz) << 4) + (byte & 15);
            if constexpr (OUT == kBF16)
              *reinterpret_cast<uint2*>(at) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
            else
              *reinterpret_cast<f32x4*>(at) = v;
          }
        }
        const int n = pass * kPassN * R + c * kPer;
        if (wide) {
#pragma unroll
          for (int q = 0; q < R / kRowsPer; ++q) {
            const int r = q * kRowsPer + r0;
            const u32x4 v = *reinterpret_cast<const u32x4*>(out + r * S::kOutRow + ((c ^ (r % kChunks)) << 4));
            const int voff = voff_c + pass * S::kOutRow, soff = (i * R + q * kRowsPer) * row_bytes;
            if (i * R + r < rows && n + kPer <= cols) {
              if (stream)
                __builtin_amdgcn_raw_buffer_store_b128(v, rc, voff, soff, kNonTemporal);
              else  // rows may start at odd bf16 elements: a global store takes any even address
                __builtin_memcpy(__builtin_assume_aligned(dst + soff + voff, 2), &v, 16);
            }
          }
          // The columns past the last whole chunk, a lane per row.
          if (tail != 0 && pass == tail_n / (kPassN * R) && lane < R && i * R + row < rows) {
            const int8_t* from = out + row * S::kOutRow + (((tail_n / kPer % kChunks) ^ swz) << 4);
            char* to = dst + (int64_t(i * R + row) * row_bytes + tail_n * kSize);
            if (tail & 8) __builtin_memcpy(__builtin_assume_aligned(to, 2), from, 8);
            if (tail & 4) __builtin_memcpy(__builtin_assume_aligned(to + (tail & 8), 2), from + (tail & 8), 4);
            if (tail & 2) __builtin_memcpy(__builtin_assume_aligned(to + (tail & 12), 2), from + (tail & 12), 2);
          }
        } else {  // offsets pass 32 bits
#pragma unroll 1
          for (int q = 0; q < R / kRowsPer; ++q) {
            const int r = q * kRowsPer + r0, m = i * R + r;
            if (m >= rows) continue;
            const int8_t* from = out + r * S::kOutRow + ((c ^ (r % kChunks)) << 4);
            char* to = dst + (int64_t(m) * P.ldc + n) * kSize;
#pragma unroll 1
            for (int e = 0; e < kPer && n + e < cols; ++e) {
              if constexpr (OUT == kBF16)
                reinterpret_cast<uint16_t*>(to)[e] = reinterpret_cast<const uint16_t*>(from)[e];
              else
                reinterpret_cast<float*>(to)[e] = reinterpret_cast<const float*>(from)[e];
            }
          }
        }
      }
    }
  }
};

template <int OUT, class S>
__global__ __launch_bounds__(64 * S::kWaves, S::kPerCu) void i8_large_kernel(const I8Params P) {
  __shared__ __align__(1024) int8_t smem[S::kLds];
  const uint32_t n_lines = uint32_t(P.K / kDepth), n_kt = n_lines < 2 ? 2 : n_lines;
  // A grid with fewer workgroups than tiles: each XCD takes a contiguous
  // range of tiles, its workgroups consecutive ones of it at a time.
  uint32_t tile = xcd_tile(gridDim.x), tile_end = tile + 1, tile_step = 1;
  if (gridDim.x != P.n_tiles) {
    const uint32_t x = blockIdx.x % 8;
    tile = uint32_t(uint64_t(P.n_tiles) * x / 8) + blockIdx.x / 8;
    tile_end = uint32_t(uint64_t(P.n_tiles) * (x + 1) / 8);
    tile_step = gridDim.x / 8;
  }
  if (tile >= tile_end) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  LargeTile<OUT, S> T{P, lane, wave, wave >> 1, wave & 1};
  T.lanes();
  int8_t* p0 = smem;
  int8_t* p1 = smem + S::kStageBytes;
  T.aim(tile);
  T.load_stage(p0, 0);
  T.load_stage(p1, 1);
  wait_loads<S::kLoads>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  T.read(0, p0, 0);
  for (;;) {
#pragma unroll
    for (int i = 0; i < S::MB; ++i)
#pragma unroll
      for (int j = 0; j < S::NB; ++j) T.acc[i][j] = i32x16{};
    uint32_t kt = 0;
    if (n_kt & 1) {  // an odd number of stages: one ahead of the pairs
      T.stage(p0, p1, 2);
      int8_t* p = p0;
      p0 = p1;
      p1 = p;
      kt = 1;
    }
    // After the last tile the loads run once more on it, into buffers that nobody reads.
    const uint32_t next = tile + tile_step < tile_end ? tile + tile_step : tile;
    T.run(p0, p1, smem + 2 * S::kStageBytes + wave * S::kOutBytes, n_kt, kt, tile, next);
    tile += tile_step;
    if (tile >= tile_end) break;
  }
  wait_loads<0>();  // the buffers stay this workgroup's until the last load has landed
}

// The 128 x 128 tile for grids that give a CU one workgroup at most, where
// only the wave itself can hide its latencies: four stages in LDS, three of
// them on their way, and the operands of a whole stage read into registers
// while the previous one is multiplied.  1024 x 2048 x 4096, 16.1 us: 256 tiles
// are one round whose first loads (3.5 us with the launch) and stores (2.5)
// nothing covers.
template <int OUT, class S>
struct DeepTile : LargeTile<OUT, S> {
  using T = LargeTile<OUT, S>;
  i32x4 a[2][S::KS][S::MB], b[2][S::KS][S::NB];

  __device__ __forceinline__ void read_stage(int set, const int8_t* __restrict__ src) {
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) {
      const int8_t* pa = src + T::wm * (S::MB * S::R * kDepth) + T::roff[ks];
      const int8_t* pb = src + (S::kM + T::wn * S::NB * S::R) * kDepth + T::roff[ks];
#pragma unroll
      for (int i = 0; i < S::MB; ++i) a[set][ks][i] = *reinterpret_cast<const i32x4*>(pa + i * S::R * kDepth);
#pragma unroll
      for (int j = 0; j < S::NB; ++j) b[set][ks][j] = *reinterpret_cast<const i32x4*>(pb + j * S::R * kDepth);
    }
  }
  // Waits for the oldest of the stages on their way, of which `newer` came after it.
  __device__ __forceinline__ void wait_oldest(uint32_t newer) {
    if (newer >= 3)
      wait_loads<3 * S::kLoads>();
    else if (newer == 2)
      wait_loads<2 * S::kLoads>();
    else if (newer == 1)
      wait_loads<S::kLoads>();
    else
      wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  // Stage s of n, whose operands are in set SET: every wave has read it, so its buffer takes stage s + 4.
  template <int SET>
  __device__ __forceinline__ void stage(int8_t* __restrict__ cur, int8_t* __restrict__ nxt, uint32_t s,
                                        uint32_t n) {
    const uint32_t left = n - s;
    wait_oldest(left >= 4 ? 2 : (left == 3 ? 1 : 0));
    if (left > 4) T::load_stage(cur, s + 4);
    read_stage(SET ^ 1, nxt);
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks)
#pragma unroll
      for (int i = 0; i < S::MB; ++i)
#pragma unroll
        for (int j = 0; j < S::NB; ++j)
          T::acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[SET][ks][j], a[SET][ks][i], T::acc[i][j], 0, 0, 0);
#pragma unroll
    for (int q = 0; q < S::KS * (S::MB + S::NB); ++q) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // an LDS read
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
    }
  }
  __device__ __forceinline__ void run(int8_t* __restrict__ p0, int8_t* __restrict__ p1,
                                      int8_t* __restrict__ p2, int8_t* __restrict__ p3, uint32_t n,
                                      typename T::template States<S::MB, S::NB>& st, uint32_t tile) {
    T::load_stage(p0, 0);
    if (n > 1) T::load_stage(p1, 1);
    if (n > 2) T::load_stage(p2, 2);
    if (n > 3) T::load_stage(p3, 3);
    if constexpr (is_step(OUT)) T::load_states(st, tile, 0, 0);
    wait_oldest(n - 1);
    read_stage(0, p0);
    for (uint32_t s = 0; s < n; s += 4) {
      stage<0>(p0, p1, s, n);
      if (s + 1 < n) stage<1>(p1, p2, s + 1, n);
      if (s + 2 < n) stage<0>(p2, p3, s + 2, n);
      if (s + 3 < n) stage<1>(p3, p0, s + 3, n);
    }
  }
};

template <int OUT, class S>
__global__ __launch_bounds__(64 * S::kWaves, 1) void i8_deep_kernel(const I8Params P) {
  // A wave's sums (step) or its results of 32 rows at a time, where the stages were.
  constexpr int kOut = is_step(OUT) ? S::MB * S::NB * S::R * 128 : S::kOutBytes;
  static_assert(S::kWaves * kOut <= 4 * S::kStageBytes);
  __shared__ __align__(1024) int8_t smem[4 * S::kStageBytes];
  const uint32_t tile = xcd_tile(gridDim.x);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  DeepTile<OUT, S> T{P, lane, wave, wave >> 1, wave & 1};
  T.lanes();
  T.aim(tile);
#pragma unroll
  for (int i = 0; i < S::MB; ++i)
#pragma unroll
    for (int j = 0; j < S::NB; ++j) T.acc[i][j] = i32x16{};
  typename LargeTile<OUT, S>::template States<S::MB, S::NB> st;
  T.run(smem, smem + S::kStageBytes, smem + 2 * S::kStageBytes, smem + 3 * S::kStageBytes, uint32_t(P.K / kDepth), st,
        tile);
  __syncthreads();  // every wave has read the last stage
  if constexpr (is_step(OUT))
    T.update(smem + wave * kOut, st, 0, 0);
  else
    T.store(smem + wave * kOut, tile);
}

template <int OUT>
void set_tiles(I8Params& P, int64_t rows, int64_t cols) {
  const int64_t n = is_step(OUT) ? 2 * P.D_h : P.N;
  P.tiles_m = uint32_t((P.M + rows - 1) / rows);
  P.tiles_n = uint32_t((n + cols - 1) / cols);
  P.n_tiles = P.tiles_m * P.tiles_n;
}

template <int OUT, int MT, int NT>
void narrow(I8Params& P, hipStream_t stream) {
  set_tiles<OUT>(P, 16 * MT, 16 * NT);
  hipLaunchKernelGGL((i8_narrow_kernel<OUT, MT, NT>), dim3(P.n_tiles), dim3(64 * kSplitWaves), 0,
                     stream, P);
}

template <int OUT>
void deep(I8Params& P, hipStream_t stream) {
  using S = LargeShape<2, 2>;
  set_tiles<OUT>(P, S::kM, S::kN);
  hipLaunchKernelGGL((i8_deep_kernel<OUT, S>), dim3(P.n_tiles), dim3(64 * S::kWaves), 0, stream, P);
}

template <int OUT, class S>
void large(I8Params& P, hipStream_t stream) {
  set_tiles<OUT>(P, S::kM, S::kN);
  const uint32_t most = kCus * S::kPerCu;
  hipLaunchKernelGGL((i8_large_kernel<OUT, S>), dim3(P.n_tiles < most ? P.n_tiles : most),
                     dim3(64 * S::kWaves), 0, stream, P);
}

// What the kernels' 32-bit offsets and one launch's grid allow.
template <int OUT>
sr_status check_sizes(const I8Params& P) {
  const int64_t n = is_step(OUT) ? 2 * P.D_h : P.N;
  if (P.M > kMaxBlocks256 || n > kMaxBlocks256 || ((P.M + 127) / 128) * ((n + 127) / 128) > kMaxBlocks256)
    return fail(SR_ERR_UNSUPPORTED, "8-bit product of %lld x %lld results too large for one launch",
                (long long)P.M, (long long)n);
  constexpr int64_t kMaxStride = int64_t(1) << 23;
  if (P.lda > kMaxStride || P.ldb > kMaxStride)
    return fail(SR_ERR_UNSUPPORTED, "rows of codes %lld bytes apart are too far apart",
                (long long)(P.lda > P.ldb ? P.lda : P.ldb));
  if (is_step(OUT) && (P.D_h > kMaxStride / 2 || n * P.ldb > int64_t(0xFFFFFFFF)))
    return fail(SR_ERR_UNSUPPORTED, "8-bit weights of %lld x %lld are too large for a step",
                (long long)n, (long long)P.ldb);
  return SR_OK;
}

sr_status launched() {
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(SR_ERR_HIP, "8-bit product launch: %s", hipGetErrorString(err));
  return SR_OK;
}

// Which kernel.  Measured in us (one launch in a replayed graph, weights from
// four alternating buffers; narrow 64 x 64 / 32 x 32 / 16 x 32, deep and
// persistent 128 x 128, 256 x 256):
//   M x K x N          64x64  32x32  16x32  deep  128x128  256x256   (fp32 results)
//   32 x 2048 x 4096     6.4    3.9    3.6     -     13.0     29.0
//   256 x 2048 x 2048    6.6    5.1    6.6     -     11.1     30.8
//   256 x 2048 x 4096    7.4    9.2   11.6  12.8     14.0     31.2
//   512 x 2048 x 4096   12.7   15.3   19.4  13.6     14.6     31.3
//   1024 x 2048 x 4096  22.9   26.8   34.7  16.1     17.3     31.5
//   8192 x 1024 x 2048  70.3      -      -  37.5     30.5     29.4
//   20000 x 2048 x 1000    -      -      -     -     56.3     68.5
//   131072 x 512 x 1024    -      -      -     -      188      140
// (a step with its quantisation, D = 2048: 512 streams 17.6 in 64 x 64, 19.0
// deep; 640 streams 23.9, 19.7).  So: 128 x 128 tiles where they are more than
// half as many as there are CUs, in the deep form while a CU has one at most;
// below that the largest narrow tile that still gives every CU one.  256 x 256
// tiles do an area's work in about 5/6 of the time, so they are taken where
// they need at most 6/5 of the rounds (one round alone only with a depth that
// carries it).
template <int OUT>
sr_status launch(I8Params P, hipStream_t stream, bool check_only) {
  const sr_status st = check_sizes<OUT>(P);
  if (st != SR_OK || check_only) return st;
  const int64_t n = is_step(OUT) ? 2 * P.D_h : P.N;
  auto tiles = [&](int64_t rows, int64_t cols) { return ((P.M + rows - 1) / rows) * ((n + cols - 1) / cols); };
  const int64_t t128 = tiles(128, 128), t256 = tiles(256, 256);
  const int64_t rounds128 = (t128 + 2 * kCus - 1) / (2 * kCus), rounds256 = (t256 + kCus - 1) / kCus;
  // (The deep form wants a stage; without any depth the persistent one stores zeros, and
  // 64 x 64 tiles of the largest results would be more than one launch holds.)
  if (t128 > (P.K > 0 ? kCus / 2 : kCus)) {
    if (t128 <= kCus)
      deep<OUT>(P, stream);
    else if (!is_step(OUT) && 5 * rounds256 <= 3 * rounds128 && (rounds256 > 1 || P.K >= 1024))
      large<is_step(OUT) ? kF32 : OUT, LargeShape<4, 4>>(P, stream);
    else
      large<OUT, LargeShape<2, 2>>(P, stream);
  } else if (tiles(64, 64) >= kCus) {
    narrow<OUT, 4, 4>(P, stream);
  } else if (tiles(32, 32) >= kCus) {
    narrow<OUT, 2, 2>(P, stream);
  } else {
    narrow<OUT, 1, 2>(P, stream);
  }
  return launched();
}

template <int OUT>
sr_status launch_tokens(I8Params P, const Tokens& x, hipStream_t stream, bool check_only) {
  P.X = x.x;
  P.Kx = int(x.K);
  const sr_status st = check_sizes<OUT>(P);
  if (st != SR_OK || check_only) return st;
  set_tiles<OUT>(P, 16, 16);
  const dim3 grid{P.n_tiles}, block{64 * kSplitWaves};
  auto run = [&](auto* kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, P); };
  const bool shallow = P.K <= kMaxTokenDepth / 4;
  if constexpr (is_step(OUT)) {  // the rows of a product are states, in fp32
    if (x.dtype == SR_BF16) {
      shallow ? run(i8_token_kernel<OUT, uint16_t, kMaxTokenDepth / 4>)
              : run(i8_token_kernel<OUT, uint16_t, kMaxTokenDepth>);
      return launched();
    }
  }
  shallow ? run(i8_token_kernel<OUT, float, kMaxTokenDepth / 4>)
          : run(i8_token_kernel<OUT, float, kMaxTokenDepth>);
  return launched();
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

// Whether the rows are few and short enough for the token kernel, and made of
// whole dwords.
bool tokens_apply(int64_t M, int64_t K, const void* x, sr_dtype dtype) {
  return M <= kMaxTokens && K > 0 && K <= kMaxTokenDepth &&
         aligned(x, 4) && (dtype == SR_F32 || K % 2 == 0);
}

sr_status launch_gemm_i8(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda,
                         const float* a_scale, const int8_t* B, int64_t ldb, const float* b_scale,
                         void* C, int64_t ldc, sr_dtype c_dtype, hipStream_t stream,
                         bool check_only, const Tokens* tokens) {
  if (M == 0 || N == 0) return SR_OK;
  I8Params P{};
  P.M = M; P.N = N; P.K = K;
  P.A = A; P.lda = lda; P.a_scale = a_scale;
  P.B = B; P.ldb = ldb; P.b_scale = b_scale;
  P.C = C; P.ldc = ldc;
  const int64_t row_bytes = ldc * (c_dtype == SR_BF16 ? 2 : 4);
  P.lines = row_bytes % 128 == 0 && aligned(C, 128);
  if (tokens != nullptr)
    return c_dtype == SR_BF16 ? launch_tokens<kBF16>(P, *tokens, stream, check_only)
                              : launch_tokens<kF32>(P, *tokens, stream, check_only);
  return c_dtype == SR_BF16 ? launch<kBF16>(P, stream, check_only) : launch<kF32>(P, stream, check_only);
}

sr_status launch_step_i8(int64_t Bsz, int64_t K, int64_t D_h, const int8_t* x, const float* x_scale,
                         const int8_t* W_in, const float* w_scale, const float* h_prev,
                         float* h_next, hipStream_t stream, const StepDecay* decay,
                         bool check_only, const Tokens* tokens) {
  if (Bsz == 0 || D_h == 0) return SR_OK;
  I8Params P{};
  P.M = Bsz; P.N = 2 * D_h; P.K = K;
  P.A = x; P.lda = K; P.a_scale = x_scale;
  P.B = W_in; P.ldb = K; P.b_scale = w_scale;
  P.D_h = D_h; P.h_prev = h_prev; P.h_next = h_next;
  if (decay != nullptr) {
    P.rate = decay->rate;
    P.gap = decay->gap;
    P.log1p_gap = decay->log1p_gap;
    P.saturated = decay->saturated;
  }
  if (tokens != nullptr)
    return decay != nullptr ? launch_tokens<kStepDecay>(P, *tokens, stream, check_only)
                            : launch_tokens<kStep>(P, *tokens, stream, check_only);
  return decay != nullptr ? launch<kStepDecay>(P, stream, check_only) : launch<kStep>(P, stream, check_only);
}

}  // namespace sr
