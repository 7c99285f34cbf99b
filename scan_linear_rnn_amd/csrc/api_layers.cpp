// C ABI entry points of the selective scan, the short convolution and the norm:
// argument validation, workspace carving, launches (as in api.cpp: every check
// runs before anything is enqueued, and without a HIP call).

#include "api_util.hpp"

namespace sr {
namespace {

constexpr int64_t kMost = int64_t(1) << 40;  // of any size

// A size with what is added to it, where that cannot overflow (else it stays too large).
int64_t padded(int64_t size, int64_t more) { return size > kMost ? size : size + more; }

bool sizes_ok(std::initializer_list<int64_t> sizes) {
  int64_t n = 16;  // bytes per element, with room to spare
  for (int64_t s : sizes) {
    if (s < 0 || s > kMost) return false;
    if (!mul_ok(n, s > 0 ? s : 1, &n)) return false;
  }
  return true;
}

// The work-items of a launch fit one grid.
sr_status check_grid(int64_t blocks, int64_t threads) {
  if (blocks > int64_t(0xFFFFFFFF) / threads)
    return fail(SR_ERR_UNSUPPORTED, "%lld workgroups exceed one launch's grid", (long long)blocks);
  return SR_OK;
}

struct Area {
  const void* p;
  int64_t bytes;
};
bool overlaps_any(Area a, std::initializer_list<Area> others) {
  for (const Area& o : others)
    if (overlap(a.p, a.bytes, o.p, o.bytes)) return true;
  return false;
}
// Rows of `width` elements ld apart, of sizes that were checked.
Area rows(const void* p, int64_t n, int64_t ld, int64_t width, sr_dtype t) {
  return {p, n > 0 && width > 0 ? ((n - 1) * ld + width) * int64_t(elem_size(t)) : 0};
}

// ------------------------------------------------------------- selective scan

// The areas of a call's workspace, each a multiple of kAlign.
struct SelectiveLayout {
  SelectivePlan plan;
  size_t ends, steps, gends, marks, parts, aparts, total;
};
SelectiveLayout selective_layout(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, bool backward) {
  SelectiveLayout L{};
  L.plan = backward ? selective_backward_plan(B, T, D, G) : selective_plan(B, T, D, G);
  const size_t channels = size_t(B) * size_t(D), c = size_t(L.plan.chunks);
  size_t at = 0;
  auto take = [&](size_t floats) {
    const size_t here = at;
    at += align_up(floats * 4, kAlign);
    return here;
  };
  if (backward || c > 1) {
    L.ends = take(c * channels * size_t(N));
    L.steps = take(c * channels);
  }
  if (backward) {
    if (c > 1) L.gends = take(c * channels * size_t(N));
    L.marks = take(size_t((T + kSelectiveTile - 1) / kSelectiveTile) * channels * size_t(N + 1));
    L.parts = take(size_t(G * L.plan.tiles_per_group) * size_t(B) * size_t(T) * 2 * size_t(selective_padded(N)));
    L.aparts = take(c * size_t(B) * size_t(N + 2) * size_t(D));
  }
  L.total = at;
  return L;
}

bool selective_sizes(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G) {
  return N >= 1 && N <= kSelectiveStates && G >= 1 && G <= kMost && sizes_ok({B, T, D, 4 * kSelectiveStates}) &&
         sizes_ok({B, T, G, 4 * kSelectiveStates}) && D % G == 0;
}

// The checks that all calls share; `tokens` is T, or 1 for a step.
sr_status check_selective(const SelectiveRequest& P, int64_t tokens, int64_t N, int64_t G) {
  SR_REQUIRE(P.B >= 0 && tokens >= 0 && P.D >= 0 && N >= 1 && G >= 1, "bad sizes (B=%lld T=%lld D=%lld N=%lld G=%lld)",
             (long long)P.B, (long long)tokens, (long long)P.D, (long long)N, (long long)G);
  if (N > kSelectiveStates)
    return fail(SR_ERR_UNSUPPORTED, "at most %d states per channel (N=%lld)", kSelectiveStates, (long long)N);
  SR_REQUIRE(P.D % G == 0, "G (%lld) must divide D (%lld)", (long long)G, (long long)P.D);
  SR_REQUIRE(selective_sizes(P.B, tokens, P.D, N, G), "tensor sizes overflow int64");
  SR_REQUIRE(is_dtype(P.dtype), "x_dtype %d unsupported", int(P.dtype));
  SR_REQUIRE(P.ld_u >= P.D && P.ld_delta >= P.D && (P.z == nullptr || P.ld_z >= P.D) && P.ld_b >= G * N &&
                 P.ld_c >= G * N,
             "row strides must be at least the rows' lengths");
  const int64_t rows_n = P.B * tokens;
  for (int64_t ld : {P.ld_u, P.ld_delta, P.z ? P.ld_z : 0, P.ld_b, P.ld_c})
    SR_REQUIRE(sizes_ok({rows_n, ld}), "tensor sizes overflow int64");
  const bool work = rows_n > 0 && P.D > 0;
  SR_REQUIRE(!work || (P.u && P.delta && P.Bm && P.Cm), "u, delta, B or C is NULL");
  SR_REQUIRE(P.D == 0 || P.A, "A is NULL");
  const size_t e = elem_size(P.dtype);
  SR_REQUIRE(aligned(P.u, e) && aligned(P.delta, e) && aligned(P.z, e) && aligned(P.Bm, e) && aligned(P.Cm, e),
             "u, delta, z, B and C must be aligned to their element size");
  SR_REQUIRE(aligned(P.A, 4) && aligned(P.skip, 4) && aligned(P.bias, 4) && aligned(P.h0, 4) && aligned(P.h_last, 4) &&
                 aligned(P.lengths, 4),
             "fp32 and int32 pointers must be 4-byte aligned");
  SR_REQUIRE(P.softplus == 0 || P.softplus == 1, "delta_softplus must be 0 or 1 (got %d)", P.softplus);
  return SR_OK;
}
// A tile's rows are addressed in 32 bits from its first one; a sequence of one token has no other.
sr_status check_rows(int64_t tokens, std::initializer_list<int64_t> apart) {
  for (int64_t ld : apart)
    if (tokens > 1 && ld > kSelectiveRow)
      return fail(SR_ERR_UNSUPPORTED, "rows are at most %lld elements apart (%lld)", (long long)kSelectiveRow, (long long)ld);
  return SR_OK;
}

// The scan's workgroups, and a thread per state where there are chunks to carry it over.
sr_status check_selective_grids(const SelectiveRequest& P, int64_t G, const SelectivePlan& plan, int threads) {
  const sr_status st = check_grid(P.B * G * plan.tiles_per_group * plan.chunks, threads);
  return st != SR_OK || plan.chunks == 1 ? st : check_grid((P.B * P.N * P.D + 255) / 256, 256);
}

Area input_area(const SelectiveRequest& P, const void* p, int64_t ld, int64_t tokens, int64_t width) {
  return rows(p, P.B * tokens, ld, width, P.dtype);
}
bool overlaps_inputs(const SelectiveRequest& P, Area out, int64_t tokens) {
  const int64_t bc = int64_t(P.G) * P.N;
  return overlaps_any(out, {input_area(P, P.u, P.ld_u, tokens, P.D), input_area(P, P.delta, P.ld_delta, tokens, P.D),
                            input_area(P, P.z, P.ld_z, tokens, P.D), input_area(P, P.Bm, P.ld_b, tokens, bc),
                            input_area(P, P.Cm, P.ld_c, tokens, bc), {P.A, 4 * P.D * P.N}, {P.skip, 4 * P.D},
                            {P.bias, 4 * P.D}});
}

void place_workspace(SelectiveRequest& P, const SelectiveLayout& L, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  auto at = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  P.tiles_per_group = int(L.plan.tiles_per_group);
  P.chunks = int(L.plan.chunks);
  P.chunk_len = L.plan.chunk_len;
  P.ends = at(L.ends);
  P.steps = at(L.steps);
  P.gends = at(L.gends);
  P.marks = at(L.marks);
  P.parts = at(L.parts);
  P.aparts = at(L.aparts);
}

// ---------------------------------------------------------------- convolution

sr_status check_conv(const ConvRequest& P, int64_t tokens, int64_t K) {
  SR_REQUIRE(P.B >= 0 && tokens >= 0 && P.D >= 0 && K >= 1, "bad sizes (B=%lld T=%lld D=%lld K=%lld)", (long long)P.B,
             (long long)tokens, (long long)P.D, (long long)K);
  if (K > kConvTaps) return fail(SR_ERR_UNSUPPORTED, "at most %d taps per channel (K=%lld)", kConvTaps, (long long)K);
  SR_REQUIRE(sizes_ok({P.B, padded(tokens, kConvTaps), P.D}) && sizes_ok({P.B * tokens, P.ld_x}), "tensor sizes overflow int64");
  SR_REQUIRE(is_dtype(P.dtype) && is_dtype(P.w_dtype), "dtype unsupported");
  SR_REQUIRE(P.ld_x >= P.D, "ld_x (%lld) must be >= D (%lld)", (long long)P.ld_x, (long long)P.D);
  SR_REQUIRE(P.x || P.B * tokens * P.D == 0, "x is NULL");
  SR_REQUIRE(P.w || P.D == 0, "w is NULL");
  const size_t e = elem_size(P.dtype), we = elem_size(P.w_dtype);
  SR_REQUIRE(aligned(P.x, e) && aligned(P.state, e) && aligned(P.last, e) && aligned(P.y, e) && aligned(P.w, we) &&
                 aligned(P.bias, we) && aligned(P.lengths, 4),
             "pointers must be aligned to their element size");
  SR_REQUIRE(P.silu == 0 || P.silu == 1, "silu must be 0 or 1 (got %d)", P.silu);
  return SR_OK;
}
int64_t conv_state_bytes(const ConvRequest& P) { return P.B * (P.K - 1) * P.D * int64_t(elem_size(P.dtype)); }

// ----------------------------------------------------------------------- norm

sr_status check_norm(int64_t M, int64_t D, sr_dtype dtype, sr_dtype r_dtype, const void* w, sr_dtype w_dtype, float eps) {
  SR_REQUIRE(M >= 0 && D >= 1, "M (%lld) must be non-negative and D (%lld) positive", (long long)M, (long long)D);
  SR_REQUIRE(sizes_ok({M, padded(D, kI8Align)}), "tensor sizes overflow int64");
  if (D > kNormWidth)
    return fail(SR_ERR_UNSUPPORTED, "rows of at most %lld elements (D=%lld)", (long long)kNormWidth, (long long)D);
  SR_REQUIRE(is_dtype(dtype) && is_dtype(r_dtype) && is_dtype(w_dtype), "dtype unsupported");
  SR_REQUIRE(w, "w is NULL");
  SR_REQUIRE(aligned(w, elem_size(w_dtype)), "w must be aligned to its element size");
  SR_REQUIRE(eps >= 0.0f && eps < 1e30f, "eps must be non-negative and finite");
  return SR_OK;
}

sr_status norm_impl(NormRequest& P, int64_t M, int64_t D, const void* x, int64_t ld_x, sr_dtype x_dtype, const void* r,
                    int64_t ld_r, sr_dtype r_dtype, const void* w, sr_dtype w_dtype, float eps, void* total,
                    std::initializer_list<Area> outs, void* stream) {
  sr_status st = check_norm(M, D, x_dtype, r ? r_dtype : x_dtype, w, w_dtype, eps);
  if (st != SR_OK) return st;
  SR_REQUIRE(ld_x >= D && (r == nullptr || ld_r >= D), "row strides must be at least D (%lld)", (long long)D);
  SR_REQUIRE(sizes_ok({M, ld_x}) && (r == nullptr || sizes_ok({M, ld_r})), "tensor sizes overflow int64");
  SR_REQUIRE(M == 0 || x, "x is NULL");
  SR_REQUIRE((r != nullptr) == (total != nullptr), "r and total go together");
  SR_REQUIRE(aligned(x, elem_size(x_dtype)) && aligned(r, elem_size(r_dtype)) && aligned(total, elem_size(r_dtype)),
             "pointers must be aligned to their element size");
  const int64_t total_bytes = M * D * int64_t(elem_size(r_dtype));
  const Area in_x = rows(x, M, ld_x, D, x_dtype), in_r = rows(r, M, ld_r, D, r_dtype);
  // A row is read whole before it is written: the sum may take the place of its own residual.
  SR_REQUIRE(!overlaps_any({total, total_bytes}, {in_x}) &&
                 (!overlap(total, total_bytes, r, in_r.bytes) || (total == r && ld_r == D)),
             "total must not overlap x, and r only as the same buffer of contiguous rows");
  for (const Area& o : outs) {
    SR_REQUIRE(!overlaps_any(o, {in_x, in_r, {total, total_bytes}, {w, D * int64_t(elem_size(w_dtype))}}),
               "outputs must not overlap inputs or each other");
    for (const Area& other : outs)
      SR_REQUIRE(&o == &other || !overlap(o.p, o.bytes, other.p, other.bytes), "outputs must not overlap each other");
  }
  P.dtype = x_dtype;
  P.r_dtype = r_dtype;
  P.w_dtype = w_dtype;
  P.M = M;
  P.D = D;
  P.x = x;
  P.r = r;
  P.ld_x = ld_x;
  P.ld_r = ld_r;
  P.w = w;
  P.eps = eps;
  P.total = total;
  P.stream = as_stream(stream);
  return M == 0 ? SR_OK : launch_norm(P);
}

}  // namespace
}  // namespace sr

using namespace sr;

extern "C" {

size_t selective_scan_forward_workspace_size(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G) {
  if (!selective_sizes(B, T, D, N, G)) return 0;
  return selective_layout(B, T, D, N, G, false).total;
}

sr_status selective_scan_forward(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, const void* u, int64_t ld_u,
                         const void* delta, int64_t ld_delta, const void* z, int64_t ld_z, const void* Bm, int64_t ld_b,
                         const void* Cm, int64_t ld_c, sr_dtype x_dtype, const float* A, const float* skip,
                         const float* delta_bias, int delta_softplus, const float* h0, const int32_t* lengths, void* y,
                         float* h_last, void* workspace, size_t workspace_bytes, void* stream) {
  clear_last_error();
  SelectiveRequest P{};
  P.dtype = x_dtype;
  P.B = B, P.T = T, P.D = D, P.N = int(N), P.G = int(G);
  P.u = u, P.delta = delta, P.z = z;
  P.ld_u = ld_u, P.ld_delta = ld_delta, P.ld_z = ld_z;
  P.Bm = Bm, P.Cm = Cm, P.ld_b = ld_b, P.ld_c = ld_c;
  P.A = A, P.skip = skip, P.bias = delta_bias, P.softplus = delta_softplus;
  P.h0 = h0, P.lengths = lengths, P.y = y, P.h_last = h_last;
  P.stream = as_stream(stream);
  sr_status st = check_selective(P, T, N, G);
  if (st == SR_OK) st = check_rows(T, {D, ld_u, ld_delta, z ? ld_z : 0, ld_b, ld_c});
  if (st != SR_OK) return st;
  const SelectiveLayout L = selective_layout(B, T, D, N, G, false);
  st = check_selective_grids(P, G, L.plan, selective_threads(N, false));
  if (st != SR_OK) return st;
  const int64_t size = int64_t(elem_size(x_dtype)), states = 4 * B * D * N;
  SR_REQUIRE(y || B * T * D == 0, "y is NULL");
  SR_REQUIRE(aligned(y, elem_size(x_dtype)), "y must be aligned to its element size");
  SR_REQUIRE(!overlaps_inputs(P, {y, size * B * T * D}, T) && !overlaps_inputs(P, {h_last, states}, T) &&
                 !overlaps_any({y, size * B * T * D}, {{h0, states}, {h_last, states}}) &&
                 !overlaps_any({h_last, states}, {{h0, states}}),
             "outputs must not overlap inputs or each other");
  st = check_workspace(workspace, workspace_bytes, L.total);
  if (st != SR_OK) return st;
  if (B == 0 || D == 0) return SR_OK;
  place_workspace(P, L, workspace);
  P.marks = nullptr;
  return launch_selective_scan(P);
}

size_t selective_scan_backward_workspace_size(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G) {
  if (!selective_sizes(B, T, D, N, G)) return 0;
  return selective_layout(B, T, D, N, G, true).total;
}

sr_status selective_scan_backward(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, const void* u, int64_t ld_u,
                                  const void* delta, int64_t ld_delta, const void* z, int64_t ld_z, const void* Bm,
                                  int64_t ld_b, const void* Cm, int64_t ld_c, sr_dtype x_dtype, const float* A,
                                  const float* skip, const float* delta_bias, int delta_softplus, const float* h0,
                                  const int32_t* lengths, const void* dy, int64_t ld_dy, const float* dh_last, void* du,
                                  void* ddelta, void* dz, void* dB, void* dC, float* dA, float* dskip, float* ddelta_bias,
                                  float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
  clear_last_error();
  SelectiveRequest P{};
  P.dtype = x_dtype;
  P.B = B, P.T = T, P.D = D, P.N = int(N), P.G = int(G);
  P.u = u, P.delta = delta, P.z = z;
  P.ld_u = ld_u, P.ld_delta = ld_delta, P.ld_z = ld_z;
  P.Bm = Bm, P.Cm = Cm, P.ld_b = ld_b, P.ld_c = ld_c;
  P.A = A, P.skip = skip, P.bias = delta_bias, P.softplus = delta_softplus;
  P.h0 = h0, P.lengths = lengths;
  P.dy = dy, P.ld_dy = ld_dy, P.dh_last = dh_last;
  P.du = du, P.ddelta = ddelta, P.dz = dz, P.dB = dB, P.dC = dC;
  P.dA = dA, P.dskip = dskip, P.dbias = ddelta_bias, P.dh0 = dh0;
  P.stream = as_stream(stream);
  sr_status st = check_selective(P, T, N, G);
  if (st != SR_OK) return st;
  const size_t e = elem_size(x_dtype);
  const int64_t n = B * T * D;
  SR_REQUIRE(ld_dy >= D && sizes_ok({B * T, ld_dy}), "ld_dy (%lld) must be >= D (%lld) and fit int64", (long long)ld_dy,
             (long long)D);
  st = check_rows(T, {D, ld_u, ld_delta, z ? ld_z : 0, ld_b, ld_c, ld_dy});
  if (st != SR_OK) return st;
  SR_REQUIRE(n == 0 || (dy && du && ddelta && dB && dC), "dy, du, ddelta, dB and dC are required");
  SR_REQUIRE(D == 0 || dA, "dA is required");
  SR_REQUIRE((z != nullptr) == (dz != nullptr) || n == 0, "z and dz go together");
  SR_REQUIRE(aligned(dy, e) && aligned(du, e) && aligned(ddelta, e) && aligned(dz, e) && aligned(dB, e) && aligned(dC, e),
             "dy and the gradients must be aligned to their element size");
  SR_REQUIRE(aligned(dh_last, 4) && aligned(dA, 4) && aligned(dskip, 4) && aligned(ddelta_bias, 4) && aligned(dh0, 4),
             "fp32 pointers must be 4-byte aligned");
  const int64_t x = int64_t(e) * n, bc = int64_t(e) * B * T * G * N, states = 4 * B * D * N;
  const Area outs[] = {{du, x},           {ddelta, x},    {dz, x},          {dB, bc},     {dC, bc},
                       {dA, 4 * D * N}, {dskip, 4 * D}, {ddelta_bias, 4 * D}, {dh0, states}};
  for (const Area& o : outs) {
    SR_REQUIRE(!overlaps_inputs(P, o, T) && !overlaps_any(o, {rows(dy, B * T, ld_dy, D, x_dtype), {h0, states}, {dh_last, states}}),
               "outputs must not overlap inputs");
    for (const Area& other : outs)
      SR_REQUIRE(&o == &other || !overlap(o.p, o.bytes, other.p, other.bytes), "outputs must not overlap each other");
  }
  const SelectiveLayout L = selective_layout(B, T, D, N, G, true);
  st = check_workspace(workspace, workspace_bytes, L.total);
  if (st != SR_OK) return st;
  st = check_selective_grids(P, G, L.plan, selective_threads(N, true));
  if (st == SR_OK) st = check_grid((B * T * G * 2 * selective_padded(N) + 255) / 256, 256);
  if (st == SR_OK) st = check_grid(((N + 2) * D + 63) / 64, 1024);
  if (st != SR_OK) return st;
  if (D == 0 && (B * T == 0 || (!dB && !dC))) return SR_OK;
  place_workspace(P, L, workspace);
  return launch_selective_backward(P);
}

sr_status selective_step(int64_t B, int64_t D, int64_t N, int64_t G, const void* u, int64_t ld_u, const void* delta,
                         int64_t ld_delta, const void* z, int64_t ld_z, const void* Bm, int64_t ld_b, const void* Cm,
                         int64_t ld_c, sr_dtype x_dtype, const float* A, const float* skip, const float* delta_bias,
                         int delta_softplus, const float* h_prev, float* h_next, void* y, void* stream) {
  clear_last_error();
  SelectiveRequest P{};
  P.dtype = x_dtype;
  P.B = B, P.T = 1, P.D = D, P.N = int(N), P.G = int(G);
  P.u = u, P.delta = delta, P.z = z;
  P.ld_u = ld_u, P.ld_delta = ld_delta, P.ld_z = ld_z;
  P.Bm = Bm, P.Cm = Cm, P.ld_b = ld_b, P.ld_c = ld_c;
  P.A = A, P.skip = skip, P.bias = delta_bias, P.softplus = delta_softplus;
  P.h0 = h_prev, P.h_last = h_next, P.y = y;
  P.stream = as_stream(stream);
  sr_status st = check_selective(P, 1, N, G);
  if (st != SR_OK) return st;
  const int64_t size = int64_t(elem_size(x_dtype)), states = 4 * B * D * N;
  SR_REQUIRE((y && h_next) || B * D == 0, "y or h_next is NULL");
  SR_REQUIRE(aligned(y, elem_size(x_dtype)), "y must be aligned to its element size");
  SR_REQUIRE(h_next == h_prev || !overlap(h_next, states, h_prev, states),
             "h_next must be the same buffer as h_prev or not overlap it");
  SR_REQUIRE(!overlaps_inputs(P, {y, size * B * D}, 1) && !overlaps_inputs(P, {h_next, states}, 1) &&
                 !overlaps_any({y, size * B * D}, {{h_prev, states}, {h_next, states}}),
             "outputs must not overlap inputs or each other");
  st = check_grid(selective_step_blocks(B, D, N), 256);
  if (st != SR_OK) return st;
  if (B == 0 || D == 0) return SR_OK;
  return launch_selective_step(P);
}

sr_status causal_conv_forward(int64_t B, int64_t T, int64_t D, int64_t K, const void* x, int64_t ld_x, sr_dtype x_dtype,
                      const void* w, const void* bias, sr_dtype w_dtype, int silu, const void* state,
                      const int32_t* lengths, void* y, void* last, void* stream) {
  clear_last_error();
  ConvRequest P{};
  P.dtype = x_dtype, P.w_dtype = w_dtype;
  P.B = B, P.T = T, P.D = D, P.K = int(K);
  P.x = x, P.ld_x = ld_x, P.w = w, P.bias = bias, P.silu = silu;
  P.state = state, P.lengths = lengths, P.y = y, P.last = last;
  P.stream = as_stream(stream);
  sr_status st = check_conv(P, T, K);
  if (st != SR_OK) return st;
  const ConvPlan plan = conv_plan(B, T, D, x_dtype, false);
  P.run_len = plan.run_len;
  P.runs = plan.runs;
  st = check_grid((conv_threads(P) + 255) / 256, 256);
  if (st != SR_OK) return st;
  const int64_t size = int64_t(elem_size(x_dtype)), kept = conv_state_bytes(P), out = size * B * T * D;
  SR_REQUIRE(y || B * T * D == 0, "y is NULL");
  const int64_t we = int64_t(elem_size(w_dtype));
  const Area in = rows(x, B * T, ld_x, D, x_dtype), wa{w, we * D * K}, ba{bias, we * D};
  SR_REQUIRE(!overlaps_any({y, out}, {in, {state, kept}, {last, kept}, wa, ba}) &&
                 !overlaps_any({last, kept}, {in, {state, kept}, wa, ba}),
             "outputs must not overlap inputs or each other");
  if (B == 0 || D == 0) return SR_OK;
  return launch_conv(P);
}

size_t causal_conv_backward_workspace_size(int64_t B, int64_t T, int64_t D, int64_t K, sr_dtype x_dtype) {
  if (K < 1 || K > kConvTaps || !is_dtype(x_dtype) || !sizes_ok({B, T < 0 ? -1 : padded(T, kConvTaps), D, kConvTaps + 1})) return 0;
  return align_up(size_t(B * conv_plan(B, T, D, x_dtype, true).runs) * size_t(K + 1) * size_t(D) * 4, kAlign);
}

sr_status causal_conv_backward(int64_t B, int64_t T, int64_t D, int64_t K, const void* x, int64_t ld_x, sr_dtype x_dtype,
                               const void* w, const void* bias, sr_dtype w_dtype, int silu, const void* state,
                               const int32_t* lengths, const void* dy, int64_t ld_dy, const void* dlast, void* dx,
                               float* dw, float* dbias, void* dstate, void* workspace, size_t workspace_bytes,
                               void* stream) {
  clear_last_error();
  ConvRequest P{};
  P.dtype = x_dtype, P.w_dtype = w_dtype;
  P.B = B, P.T = T, P.D = D, P.K = int(K);
  P.x = x, P.ld_x = ld_x, P.w = w, P.bias = bias, P.silu = silu;
  P.state = state, P.lengths = lengths;
  P.dy = dy, P.ld_dy = ld_dy, P.dlast = dlast, P.dx = dx, P.dw = dw, P.dbias = dbias, P.dstate = dstate;
  P.stream = as_stream(stream);
  sr_status st = check_conv(P, T, K);
  if (st != SR_OK) return st;
  const ConvPlan plan = conv_plan(B, T, D, x_dtype, true);
  P.run_len = plan.run_len;
  P.runs = plan.runs;
  st = check_grid((conv_backward_threads(P) + 255) / 256, 256);
  if (st == SR_OK) st = check_grid(((K + 1) * D + 63) / 64, 1024);
  if (st != SR_OK) return st;
  const size_t e = elem_size(x_dtype);
  const int64_t n = B * T * D, kept = conv_state_bytes(P), we = int64_t(elem_size(w_dtype));
  SR_REQUIRE(ld_dy >= D && sizes_ok({B * T, ld_dy}), "ld_dy (%lld) must be >= D (%lld) and fit int64", (long long)ld_dy,
             (long long)D);
  SR_REQUIRE(n == 0 || (dy && dx), "dy and dx are required");
  SR_REQUIRE(D == 0 || dw, "dw is required");
  SR_REQUIRE(aligned(dy, e) && aligned(dlast, e) && aligned(dx, e) && aligned(dstate, e) && aligned(dw, 4) &&
                 aligned(dbias, 4),
             "pointers must be aligned to their element size");
  const Area ins[] = {rows(x, B * T, ld_x, D, x_dtype), rows(dy, B * T, ld_dy, D, x_dtype), {state, kept}, {dlast, kept},
                      {w, we * D * K}, {bias, we * D}};
  const Area outs[] = {{dx, int64_t(e) * n}, {dw, 4 * D * K}, {dbias, 4 * D}, {dstate, kept}};
  for (const Area& o : outs) {
    for (const Area& i : ins) SR_REQUIRE(!overlap(o.p, o.bytes, i.p, i.bytes), "outputs must not overlap inputs");
    for (const Area& other : outs)
      SR_REQUIRE(&o == &other || !overlap(o.p, o.bytes, other.p, other.bytes), "outputs must not overlap each other");
  }
  st = check_workspace(workspace, workspace_bytes, causal_conv_backward_workspace_size(B, T, D, K, x_dtype));
  if (st != SR_OK) return st;
  P.parts = static_cast<float*>(workspace);
  if (D == 0) return SR_OK;
  return launch_conv_backward(P);
}

sr_status causal_conv_step(int64_t B, int64_t D, int64_t K, const void* x, int64_t ld_x, sr_dtype x_dtype, const void* w,
                           const void* bias, sr_dtype w_dtype, int silu, const void* state, void* state_next, void* y,
                           void* stream) {
  clear_last_error();
  ConvRequest P{};
  P.dtype = x_dtype, P.w_dtype = w_dtype;
  P.B = B, P.T = 1, P.D = D, P.K = int(K);
  P.x = x, P.ld_x = ld_x, P.w = w, P.bias = bias, P.silu = silu;
  P.state = state, P.last = state_next, P.y = y;
  P.stream = as_stream(stream);
  sr_status st = check_conv(P, 1, K);
  if (st != SR_OK) return st;
  const int64_t size = int64_t(elem_size(x_dtype)), kept = conv_state_bytes(P), we = int64_t(elem_size(w_dtype));
  SR_REQUIRE(y || B * D == 0, "y is NULL");
  SR_REQUIRE(state_next || kept == 0, "state_next is NULL");
  const Area in = rows(x, B, ld_x, D, x_dtype), wa{w, we * D * K}, ba{bias, we * D};
  SR_REQUIRE(state_next == state || !overlap(state_next, kept, state, kept),
             "state_next must be the same buffer as state or not overlap it");
  SR_REQUIRE(!overlaps_any({y, size * B * D}, {in, {state, kept}, {state_next, kept}, wa, ba}) &&
                 !overlaps_any({state_next, kept}, {in, wa, ba}),
             "outputs must not overlap inputs or each other");
  st = check_grid((conv_step_threads(P) + 255) / 256, 256);
  if (st != SR_OK) return st;
  if (B == 0 || D == 0) return SR_OK;
  return launch_conv_step(P);
}

sr_status rms_norm_forward(int64_t M, int64_t D, const void* x, int64_t ld_x, sr_dtype x_dtype, const void* r, int64_t ld_r,
                   sr_dtype r_dtype, const void* w, sr_dtype w_dtype, float eps, void* total, void* y, void* stream) {
  clear_last_error();
  NormRequest P{};
  SR_REQUIRE(y || M <= 0, "y is NULL");
  SR_REQUIRE(aligned(y, elem_size(x_dtype)), "y must be aligned to its element size");
  P.y = y;
  int64_t n;
  SR_REQUIRE(M >= 0 && D >= 0 && prod3(M, D, 16, &n), "sizes must be non-negative and fit int64");
  return norm_impl(P, M, D, x, ld_x, x_dtype, r, ld_r, r_dtype, w, w_dtype, eps, total,
                   {{y, M * D * int64_t(elem_size(x_dtype))}}, stream);
}

sr_status rms_norm_quantize(int64_t M, int64_t D, const void* x, int64_t ld_x, sr_dtype x_dtype, const void* r,
                            int64_t ld_r, sr_dtype r_dtype, const void* w, sr_dtype w_dtype, float eps, void* total,
                            int8_t* q, float* scale, void* stream) {
  clear_last_error();
  NormRequest P{};
  SR_REQUIRE((q && scale) || M <= 0, "q or scale is NULL");
  SR_REQUIRE(aligned(q, 16) && aligned(scale, 4), "q must be 16-byte and scale 4-byte aligned");
  int64_t n;
  SR_REQUIRE(M >= 0 && D >= 0 && D <= kMost && prod3(M, D + kI8Align, 16, &n), "sizes must be non-negative and fit int64");
  P.q = q;
  P.scale = scale;
  P.ld_q = sr::quantized_row_bytes(D);
  return norm_impl(P, M, D, x, ld_x, x_dtype, r, ld_r, r_dtype, w, w_dtype, eps, total, {{q, M * P.ld_q}, {scale, 4 * M}}, stream);
}

size_t rms_norm_backward_workspace_size(int64_t M, int64_t D) {
  if (M < 0 || D < 1 || D > kNormWidth || M > kMost) return 0;
  return align_up(size_t(norm_backward_blocks(M, D)) * size_t(D) * 4, kAlign);
}

sr_status rms_norm_backward(int64_t M, int64_t D, const void* total, int64_t ld_total, sr_dtype total_dtype, const void* w,
                            sr_dtype w_dtype, float eps, const void* dy, int64_t ld_dy, sr_dtype dy_dtype,
                            const void* dtotal, int64_t ld_dtotal, void* dx, float* dw, void* workspace,
                            size_t workspace_bytes, void* stream) {
  clear_last_error();
  sr_status st = check_norm(M, D, dy_dtype, total_dtype, w, w_dtype, eps);
  if (st != SR_OK) return st;
  SR_REQUIRE(ld_total >= D && ld_dy >= D && (dtotal == nullptr || ld_dtotal >= D), "row strides must be at least D (%lld)",
             (long long)D);
  SR_REQUIRE(sizes_ok({M, ld_total}) && sizes_ok({M, ld_dy}) && (dtotal == nullptr || sizes_ok({M, ld_dtotal})),
             "tensor sizes overflow int64");
  SR_REQUIRE(M == 0 || (total && dy && dx), "total, dy and dx are required");
  SR_REQUIRE(dw, "dw is required");
  const size_t te = elem_size(total_dtype);
  SR_REQUIRE(aligned(total, te) && aligned(dtotal, te) && aligned(dx, te) && aligned(dy, elem_size(dy_dtype)) && aligned(dw, 4),
             "pointers must be aligned to their element size");
  const Area ins[] = {rows(total, M, ld_total, D, total_dtype), rows(dy, M, ld_dy, D, dy_dtype),
                      rows(dtotal, M, ld_dtotal, D, total_dtype), {w, D * int64_t(elem_size(w_dtype))}};
  const Area da{dx, M * D * int64_t(te)}, wa{dw, 4 * D};
  for (const Area& i : ins)
    SR_REQUIRE(!overlap(da.p, da.bytes, i.p, i.bytes) && !overlap(wa.p, wa.bytes, i.p, i.bytes),
               "outputs must not overlap inputs");
  SR_REQUIRE(!overlap(da.p, da.bytes, wa.p, wa.bytes), "outputs must not overlap each other");
  st = check_workspace(workspace, workspace_bytes, rms_norm_backward_workspace_size(M, D));
  if (st != SR_OK) return st;
  NormRequest P{};
  P.dtype = dy_dtype, P.r_dtype = total_dtype, P.w_dtype = w_dtype;
  P.M = M, P.D = D, P.w = w, P.eps = eps;
  P.t = total, P.dy = dy, P.dt = dtotal;
  P.ld_t = ld_total, P.ld_dy = ld_dy, P.ld_dt = ld_dtotal;
  P.dx = dx, P.dw = dw, P.parts = static_cast<float*>(workspace);
  P.stream = as_stream(stream);
  return launch_norm_backward(P);
}

}  // extern "C"
