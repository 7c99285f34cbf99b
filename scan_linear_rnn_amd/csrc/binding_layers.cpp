// Python binding of the selective scan, the short convolution and the norm:
// marshalling only, as in binding.cpp.

#include <c10/core/DeviceGuard.h>

#include "binding_util.hpp"

namespace {

struct LayersApi {
  decltype(&::selective_scan_forward_workspace_size) scan_workspace;
  decltype(&::selective_scan_forward) scan;
  decltype(&::selective_scan_backward_workspace_size) scan_backward_workspace;
  decltype(&::selective_scan_backward) scan_backward;
  decltype(&::selective_step) step;
  decltype(&::causal_conv_forward) conv;
  decltype(&::causal_conv_backward_workspace_size) conv_backward_workspace;
  decltype(&::causal_conv_backward) conv_backward;
  decltype(&::causal_conv_step) conv_step;
  decltype(&::rms_norm_forward) norm;
  decltype(&::rms_norm_quantize) norm_quantize;
  decltype(&::rms_norm_backward_workspace_size) norm_backward_workspace;
  decltype(&::rms_norm_backward) norm_backward;
} api;

// A tensor whose dimensions from `lead` on are one row each: a view where the
// rows are evenly apart, else a copy.
struct TokenRows {
  Tensor t;
  int64_t ld = 0;
};
TokenRows token_rows(const Tensor& t, int64_t lead) {
  int64_t width = 1;
  bool even = true;
  for (int64_t i = t.dim() - 1; i >= lead; --i) {
    even = even && (t.size(i) == 1 || t.stride(i) == width);
    width *= t.size(i);
  }
  int64_t ld = 0, n = 1;  // of the rows so far, from the innermost
  for (int64_t i = lead - 1; i >= 0 && even; --i) {
    if (t.size(i) == 1) continue;
    if (n == 1)
      ld = t.stride(i);
    else
      even = t.stride(i) == ld * n;
    n *= t.size(i);
  }
  if (n <= 1) ld = width;
  if (even && ld >= width) return {t, ld};
  return {t.contiguous(), width};
}

// What a tensor of a call must be: like the first one, in type and place.
TokenRows like_first(const Tensor& t, const std::string& name, const Tensor& first, at::IntArrayRef shape, int64_t lead) {
  has_type(t, name, first.scalar_type());
  has_shape(t, name, shape);
  same_device(t, name, first);
  return token_rows(t, lead);
}
Tensor floats(const Tensor& t, const std::string& name, const Tensor& first, at::IntArrayRef shape) {
  has_type(t, name, at::kFloat);
  has_shape(t, name, shape);
  same_device(t, name, first);
  return t.contiguous();
}
MaybeTensor floats(const MaybeTensor& t, const std::string& name, const Tensor& first, at::IntArrayRef shape) {
  return t ? MaybeTensor(floats(*t, name, first, shape)) : t;
}
MaybeTensor lengths_of(const MaybeTensor& t, int64_t B, const Tensor& first) {
  if (!t) return t;
  has_type(*t, "lengths", at::kInt);
  has_shape(*t, "lengths", {B});
  same_device(*t, "lengths", first);
  return t->contiguous();
}
void has_dims(const Tensor& t, const char* name, int64_t dims) {
  if (t.dim() != dims)
    bad_value(std::string(name) + " must have " + std::to_string(dims) + " dims (got shape " + text(t.sizes()) + ")");
}

// ------------------------------------------------------------- selective scan

// The operands that the scan's calls share; `lead` leading dimensions (batch,
// and time where there is one).
struct Selective {
  sr_dtype type;
  int64_t B, T, D, N, G, lead;
  std::vector<int64_t> x_shape, bc_shape;
  TokenRows u, delta, z, Bm, Cm;
  Tensor A;
  MaybeTensor skip, bias;
  bool gated;
};
Selective selective_of(const Tensor& u, const Tensor& delta, const Tensor& A, const Tensor& B, const Tensor& C,
                       const MaybeTensor& skip, const MaybeTensor& z, const MaybeTensor& bias, int64_t lead) {
  Selective s;
  s.type = float_type(u, "u");
  has_dims(u, "u", lead + 1);
  s.lead = lead;
  s.x_shape = u.sizes().vec();
  s.B = u.size(0);
  s.T = lead == 2 ? u.size(1) : 1;
  s.D = u.size(lead);
  on_gpu(A, "A");
  has_dims(A, "A", 2);
  s.N = A.size(1);
  s.A = floats(A, "A", u, {s.D, s.N});
  on_gpu(B, "B");
  if (B.dim() != lead + 1 && B.dim() != lead + 2)
    bad_value("B must have " + std::to_string(lead + 1) + " or " + std::to_string(lead + 2) + " dims (got shape " +
              text(B.sizes()) + ")");
  s.G = B.dim() == lead + 2 ? B.size(lead) : 1;
  if (s.G < 1 || s.D % s.G)
    bad_value("the groups of B (" + std::to_string(s.G) + ") must divide the channels (" + std::to_string(s.D) + ")");
  s.bc_shape.assign(s.x_shape.begin(), s.x_shape.end() - 1);
  if (B.dim() == lead + 2) s.bc_shape.push_back(s.G);
  s.bc_shape.push_back(s.N);
  s.u = token_rows(u, lead);
  s.delta = like_first(delta, "delta", u, s.x_shape, lead);
  s.Bm = like_first(B, "B", u, s.bc_shape, lead);
  s.Cm = like_first(C, "C", u, s.bc_shape, lead);
  s.gated = z.has_value();
  if (z) s.z = like_first(*z, "z", u, s.x_shape, lead);
  s.skip = floats(skip, "skip", u, {s.D});
  s.bias = floats(bias, "delta_bias", u, {s.D});
  return s;
}
void* gate(const Selective& s) { return s.gated ? data(s.z.t) : nullptr; }

py::object call_selective_scan(const Tensor& u, const Tensor& delta, const Tensor& A, const Tensor& B, const Tensor& C,
                               const MaybeTensor& skip, const MaybeTensor& z, const MaybeTensor& bias, bool softplus,
                               const MaybeTensor& h0_in, const MaybeTensor& lengths_in, bool return_last,
                               const MaybeTensor& workspace) {
  const Selective s = selective_of(u, delta, A, B, C, skip, z, bias, 2);
  const c10::DeviceGuard guard(u.device());
  const MaybeTensor h0 = floats(h0_in, "h0", u, {s.B, s.D, s.N}), lengths = lengths_of(lengths_in, s.B, u);
  const Tensor y = make(u, s.x_shape, u.scalar_type());
  MaybeTensor last;
  if (return_last) last = make(u, {s.B, s.D, s.N}, at::kFloat);
  const Tensor ws = workspace_of(workspace, api.scan_workspace(s.B, s.T, s.D, s.N, s.G), u);
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.scan(s.B, s.T, s.D, s.N, s.G, data(s.u.t), s.u.ld, data(s.delta.t), s.delta.ld, gate(s), s.z.ld,
                  data(s.Bm.t), s.Bm.ld, data(s.Cm.t), s.Cm.ld, s.type, data<float>(s.A), data<float>(s.skip),
                  data<float>(s.bias), softplus, data<float>(h0), data<int32_t>(lengths), data(y), data<float>(last),
                  ws.data_ptr(), size_t(ws.numel()), stream_of(u));
  }
  check("selective_scan_forward", st);
  if (!return_last) return py::cast(y);
  return py::make_tuple(y, *last);
}

py::tuple call_selective_scan_backward(const Tensor& u, const Tensor& delta, const Tensor& A, const Tensor& B,
                                       const Tensor& C, const Tensor& dy_in, const MaybeTensor& skip, const MaybeTensor& z,
                                       const MaybeTensor& bias, bool softplus, const MaybeTensor& h0_in,
                                       const MaybeTensor& lengths_in, const MaybeTensor& dh_last_in,
                                       const MaybeTensor& workspace) {
  const Selective s = selective_of(u, delta, A, B, C, skip, z, bias, 2);
  const c10::DeviceGuard guard(u.device());
  const MaybeTensor h0 = floats(h0_in, "h0", u, {s.B, s.D, s.N}), lengths = lengths_of(lengths_in, s.B, u),
                    dh_last = floats(dh_last_in, "dh_last", u, {s.B, s.D, s.N});
  const TokenRows dy = like_first(dy_in, "dy", u, s.x_shape, 2);
  const at::ScalarType type = u.scalar_type();
  const Tensor du = make(u, s.x_shape, type), ddelta = make(u, s.x_shape, type), dB = make(u, s.bc_shape, type),
               dC = make(u, s.bc_shape, type), dA = make(u, {s.D, s.N}, at::kFloat);
  MaybeTensor dz, dskip, dbias, dh0;
  if (s.gated) dz = make(u, s.x_shape, type);
  if (skip) dskip = make(u, {s.D}, at::kFloat);
  if (bias) dbias = make(u, {s.D}, at::kFloat);
  if (h0) dh0 = make(u, {s.B, s.D, s.N}, at::kFloat);
  const Tensor ws = workspace_of(workspace, api.scan_backward_workspace(s.B, s.T, s.D, s.N, s.G), u);
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.scan_backward(s.B, s.T, s.D, s.N, s.G, data(s.u.t), s.u.ld, data(s.delta.t), s.delta.ld, gate(s), s.z.ld,
                           data(s.Bm.t), s.Bm.ld, data(s.Cm.t), s.Cm.ld, s.type, data<float>(s.A), data<float>(s.skip),
                           data<float>(s.bias), softplus, data<float>(h0), data<int32_t>(lengths), data(dy.t), dy.ld,
                           data<float>(dh_last), data(du), data(ddelta), data(dz), data(dB), data(dC), data<float>(dA),
                           data<float>(dskip), data<float>(dbias), data<float>(dh0), ws.data_ptr(), size_t(ws.numel()),
                           stream_of(u));
  }
  check("selective_scan_backward", st);
  return py::make_tuple(du, ddelta, dA, dB, dC, dskip, dz, dbias, dh0);
}

std::pair<Tensor, Tensor> call_selective_step(const Tensor& u, const Tensor& delta, const Tensor& A, const Tensor& B,
                                              const Tensor& C, const MaybeTensor& skip, const MaybeTensor& z,
                                              const MaybeTensor& bias, bool softplus, const MaybeTensor& h_prev,
                                              const MaybeTensor& h_next) {
  const Selective s = selective_of(u, delta, A, B, C, skip, z, bias, 1);
  const c10::DeviceGuard guard(u.device());
  if (h_prev) in_place(*h_prev, "h_prev", at::kFloat, {s.B, s.D, s.N}, u);
  if (h_next) in_place(*h_next, "h_next", at::kFloat, {s.B, s.D, s.N}, u);
  const Tensor y = make(u, s.x_shape, u.scalar_type()), h = h_next ? *h_next : make(u, {s.B, s.D, s.N}, at::kFloat);
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.step(s.B, s.D, s.N, s.G, data(s.u.t), s.u.ld, data(s.delta.t), s.delta.ld, gate(s), s.z.ld, data(s.Bm.t),
                  s.Bm.ld, data(s.Cm.t), s.Cm.ld, s.type, data<float>(s.A), data<float>(s.skip), data<float>(s.bias),
                  softplus, data<float>(h_prev), data<float>(h), data(y), stream_of(u));
  }
  check("selective_step", st);
  written(h_next);
  return {y, h};
}

// ---------------------------------------------------------------- convolution

struct Conv {
  sr_dtype type, w_type;
  int64_t B, T, D, K;
  std::vector<int64_t> x_shape, state_shape;
  TokenRows x;
  Tensor w;
  MaybeTensor bias;
};
Conv conv_of(const Tensor& x, const Tensor& w, const MaybeTensor& bias, int64_t lead) {
  Conv c;
  c.type = float_type(x, "x");
  has_dims(x, "x", lead + 1);
  c.x_shape = x.sizes().vec();
  c.B = x.size(0);
  c.T = lead == 2 ? x.size(1) : 1;
  c.D = x.size(lead);
  c.w_type = float_type(w, "weight");
  has_dims(w, "weight", 2);
  c.K = w.size(1);
  if (w.size(0) != c.D || c.K < 1) bad_value("weight must be [" + std::to_string(c.D) + ", K] (got shape " + text(w.sizes()) + ")");
  same_device(w, "weight", x);
  c.state_shape = {c.B, c.K - 1, c.D};
  c.x = token_rows(x, lead);
  c.w = w.contiguous();
  if (bias) {
    has_type(*bias, "bias", w.scalar_type());
    has_shape(*bias, "bias", {c.D});
    same_device(*bias, "bias", x);
    c.bias = bias->contiguous();
  }
  return c;
}
MaybeTensor conv_state(const MaybeTensor& t, const char* name, const Conv& c, const Tensor& x) {
  if (!t) return t;
  has_type(*t, name, x.scalar_type());
  has_shape(*t, name, c.state_shape);
  same_device(*t, name, x);
  return t->contiguous();
}

py::object call_causal_conv(const Tensor& x, const Tensor& w, const MaybeTensor& bias, bool silu, const MaybeTensor& state_in,
                            const MaybeTensor& lengths_in, bool return_last) {
  const Conv c = conv_of(x, w, bias, 2);
  const c10::DeviceGuard guard(x.device());
  const MaybeTensor state = conv_state(state_in, "state", c, x), lengths = lengths_of(lengths_in, c.B, x);
  const Tensor y = make(x, c.x_shape, x.scalar_type());
  MaybeTensor last;
  if (return_last) last = make(x, c.state_shape, x.scalar_type());
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.conv(c.B, c.T, c.D, c.K, data(c.x.t), c.x.ld, c.type, data(c.w), data(c.bias), c.w_type, silu, data(state),
                  data<int32_t>(lengths), data(y), data(last), stream_of(x));
  }
  check("causal_conv_forward", st);
  if (!return_last) return py::cast(y);
  return py::make_tuple(y, *last);
}

py::tuple call_causal_conv_backward(const Tensor& x, const Tensor& w, const Tensor& dy_in, const MaybeTensor& bias, bool silu,
                                    const MaybeTensor& state_in, const MaybeTensor& lengths_in, const MaybeTensor& dlast_in,
                                    const MaybeTensor& workspace) {
  const Conv c = conv_of(x, w, bias, 2);
  const c10::DeviceGuard guard(x.device());
  const MaybeTensor state = conv_state(state_in, "state", c, x), lengths = lengths_of(lengths_in, c.B, x),
                    dlast = conv_state(dlast_in, "dlast", c, x);
  const TokenRows dy = like_first(dy_in, "dy", x, c.x_shape, 2);
  const Tensor dx = make(x, c.x_shape, x.scalar_type()), dw = make(x, {c.D, c.K}, at::kFloat);
  MaybeTensor dbias, dstate;
  if (bias) dbias = make(x, {c.D}, at::kFloat);
  if (state) dstate = make(x, c.state_shape, x.scalar_type());
  const Tensor ws = workspace_of(workspace, api.conv_backward_workspace(c.B, c.T, c.D, c.K, c.type), x);
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.conv_backward(c.B, c.T, c.D, c.K, data(c.x.t), c.x.ld, c.type, data(c.w), data(c.bias), c.w_type, silu,
                           data(state), data<int32_t>(lengths), data(dy.t), dy.ld, data(dlast), data(dx), data<float>(dw),
                           data<float>(dbias), data(dstate), ws.data_ptr(), size_t(ws.numel()), stream_of(x));
  }
  check("causal_conv_backward", st);
  return py::make_tuple(dx, dw, dbias, dstate);
}

std::pair<Tensor, Tensor> call_causal_conv_step(const Tensor& x, const Tensor& w, const MaybeTensor& bias, bool silu,
                                                const MaybeTensor& state, const MaybeTensor& state_next) {
  const Conv c = conv_of(x, w, bias, 1);
  const c10::DeviceGuard guard(x.device());
  if (state) in_place(*state, "state", x.scalar_type(), c.state_shape, x);
  if (state_next) in_place(*state_next, "state_next", x.scalar_type(), c.state_shape, x);
  const Tensor y = make(x, c.x_shape, x.scalar_type()), next = state_next ? *state_next : make(x, c.state_shape, x.scalar_type());
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.conv_step(c.B, c.D, c.K, data(c.x.t), c.x.ld, c.type, data(c.w), data(c.bias), c.w_type, silu, data(state),
                       data(next), data(y), stream_of(x));
  }
  check("causal_conv_step", st);
  written(state_next);
  return {y, next};
}

// ----------------------------------------------------------------------- norm

struct Norm {
  Rows x, r;
  Tensor w, total;
  sr_dtype w_type;
  bool residual;
};
Tensor norm_weight(const Tensor& w, int64_t D, const Tensor& x, sr_dtype* type) {
  *type = float_type(w, "weight");
  has_shape(w, "weight", {D});
  same_device(w, "weight", x);
  return w.contiguous();
}
Norm norm_of(const Tensor& x, const Tensor& w, const MaybeTensor& residual) {
  Norm n;
  n.x = rows_of(x, "x", 0);
  n.w = norm_weight(w, n.x.width, x, &n.w_type);
  n.residual = residual.has_value();
  n.r.stride = n.r.type = 0;
  if (residual) {
    n.r = rows_of(*residual, "residual", 0);
    has_shape(*residual, "residual", x.sizes());
    same_device(*residual, "residual", x);
    n.total = make(x, x.sizes(), residual->scalar_type());
  }
  return n;
}

py::object call_rms_norm(const Tensor& x, const Tensor& w, const MaybeTensor& residual, double eps) {
  const Norm n = norm_of(x, w, residual);
  const c10::DeviceGuard guard(x.device());
  const Tensor y = make(x, x.sizes(), x.scalar_type());
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.norm(n.x.n, n.x.width, data(n.x.t), n.x.stride, n.x.type, n.residual ? data(n.r.t) : nullptr, n.r.stride,
                  n.r.type, data(n.w), n.w_type, float(eps), n.residual ? data(n.total) : nullptr, data(y), stream_of(x));
  }
  check("rms_norm_forward", st);
  if (!n.residual) return py::cast(y);
  return py::make_tuple(y, n.total);
}

py::tuple call_rms_norm_quantize(const Tensor& x, const Tensor& w, const MaybeTensor& residual, double eps) {
  const Norm n = norm_of(x, w, residual);
  const c10::DeviceGuard guard(x.device());
  std::vector<int64_t> shape(x.sizes().begin(), x.sizes().end() - 1);
  const Tensor scale = make(x, shape, at::kFloat);
  shape.push_back(stored_width(n.x.width));
  const Tensor q = make(x, shape, at::kChar);
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.norm_quantize(n.x.n, n.x.width, data(n.x.t), n.x.stride, n.x.type, n.residual ? data(n.r.t) : nullptr,
                           n.r.stride, n.r.type, data(n.w), n.w_type, float(eps), n.residual ? data(n.total) : nullptr,
                           data<int8_t>(q), data<float>(scale), stream_of(x));
  }
  check("rms_norm_quantize", st);
  if (!n.residual) return py::make_tuple(q, scale);
  return py::make_tuple(q, scale, n.total);
}

py::tuple call_rms_norm_backward(const Tensor& total, const Tensor& w, const Tensor& dy, const MaybeTensor& dtotal, double eps,
                                 const MaybeTensor& workspace) {
  const Rows t = rows_of(total, "total", 0), g = rows_of(dy, "dy", 0);
  has_shape(dy, "dy", total.sizes());
  same_device(dy, "dy", total);
  sr_dtype w_type;
  const Tensor weight = norm_weight(w, t.width, total, &w_type);
  Rows d;
  d.stride = 0;
  if (dtotal) {
    d = rows_of(*dtotal, "dtotal", 0);
    has_type(*dtotal, "dtotal", total.scalar_type());
    has_shape(*dtotal, "dtotal", total.sizes());
    same_device(*dtotal, "dtotal", total);
  }
  const c10::DeviceGuard guard(total.device());
  const Tensor dx = make(total, total.sizes(), total.scalar_type()), dw = make(total, {t.width}, at::kFloat);
  const Tensor ws = workspace_of(workspace, api.norm_backward_workspace(t.n, t.width), total);
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.norm_backward(t.n, t.width, data(t.t), t.stride, t.type, data(weight), w_type, float(eps), data(g.t), g.stride,
                           g.type, dtotal ? data(d.t) : nullptr, d.stride, data(dx), data<float>(dw), ws.data_ptr(),
                           size_t(ws.numel()), stream_of(total));
  }
  check("rms_norm_backward", st);
  return py::make_tuple(dx, dw);
}

constexpr const char* kScanDoc =
    R"(selective_scan_forward(u, delta, A, B, C, *, skip=None, z=None, delta_bias=None, delta_softplus=False, h0=None,
                       lengths=None, return_last=False, workspace=None)

The selective state space scan over [B,T,D] inputs, per channel with N states:

    dt = softplus(delta + delta_bias)  (without ``delta_softplus``: the sum itself)
    h_n = exp(dt A_n) h_n + dt u B_n,   y = (sum_n C_n h_n + skip u) silu(z)

``u``, ``delta``, ``z`` [B,T,D] and ``B``, ``C`` [B,T,N] (or [B,T,G,N]: G groups of
neighbouring channels) are fp32 or all bf16, and may be rows of a wider buffer;
``A`` [D,N], ``skip`` and ``delta_bias`` [D], the state ``h0`` [B,D,N] (None: zeros) are
fp32.  ``lengths`` [B] int32: tokens of each sequence of a padded batch; behind
them y is zero and the state stays.  N is at most 64.  Returns y in u's type, and
the last state when ``return_last``.)";
constexpr const char* kScanBackwardDoc =
    R"(selective_scan_backward(u, delta, A, B, C, dy, *, skip=None, z=None, delta_bias=None, delta_softplus=False,
                        h0=None, lengths=None, dh_last=None, workspace=None)

Gradients of ``selective_scan_forward`` for the gradients ``dy`` [B,T,D] on y and
``dh_last`` [B,D,N] on the last state: (du, ddelta, dA, dB, dC, dskip, dz,
ddelta_bias, dh0), those of the tensors in u's type, of the fp32 operands in fp32, None
for absent operands.)";
constexpr const char* kStepDoc =
    R"(selective_step(u, delta, A, B, C, *, skip=None, z=None, delta_bias=None, delta_softplus=False, h_prev=None,
               h_next=None)

One token of ``selective_scan_forward``: u, delta, z [B,D], B and C [B,N] or
[B,G,N] -> (y [B,D] in u's type, h [B,D,N] fp32).  ``h_prev`` None is the zero state;
``h_next`` may be ``h_prev`` (a step in place).)";
constexpr const char* kConvDoc =
    R"(causal_conv_forward(x, weight, bias=None, *, silu=False, state=None, lengths=None, return_last=False)

Short causal convolution over [B,T,D], a filter of K taps per channel (at most 8):
y_t = bias + sum_j weight[:, j] x_{t-K+1+j}, with ``silu`` its SiLU.  x fp32 or bf16,
``weight`` [D,K] and ``bias`` [D] of one type of the two.  ``state`` [B,K-1,D] in x's type
holds the inputs in front of the first token, oldest first (None: zeros).  ``lengths`` [B] int32: tokens of
each sequence of a padded batch; behind them y is zero.  Returns y in x's type, and
the state behind the sequence when ``return_last``.)";
constexpr const char* kConvBackwardDoc =
    R"(causal_conv_backward(x, weight, dy, bias=None, *, silu=False, state=None, lengths=None, dlast=None, workspace=None)

Gradients of ``causal_conv_forward`` for ``dy`` on y and ``dlast`` [B,K-1,D] on the
state behind the sequence: (dx in x's type, dweight and dbias in fp32, dstate in
x's type), None for absent operands.)";
constexpr const char* kConvStepDoc =
    R"(causal_conv_step(x, weight, bias=None, *, silu=False, state=None, state_next=None)

One token of ``causal_conv_forward``: x [B,D] -> (y [B,D], the state moved on by
x).  ``state_next`` may be ``state`` (a step in place).)";
constexpr const char* kNormDoc = R"(rms_norm_forward(x, weight, residual=None, *, eps=1e-6)

Root-mean-square norm of the rows (last dimension, at most 16384) of ``x`` [.., D],
fp32 or bf16: y = t / sqrt(mean(t^2) + eps) * weight in x's type.  With ``residual`` (of
x's shape, fp32 or bf16) t is x + residual, rounded to the residual's type, and
(y, t) is returned: t is the next residual.)";
constexpr const char* kNormQuantizeDoc = R"(rms_norm_quantize(x, weight, residual=None, *, eps=1e-6)

``rms_norm_forward`` with y as 8-bit codes and a scale per row, for matmul_i8:
(q [.., quantized_row_bytes(D)] int8, scale [..] fp32), as quantize_rows makes them but
of the fp32 values; with ``residual`` also t.)";
constexpr const char* kNormBackwardDoc =
    R"(rms_norm_backward(total, weight, dy, *, dtotal=None, eps=1e-6, workspace=None)

Gradients of ``rms_norm_forward``: ``total`` is the t it returned (x without a
residual), ``dy`` the gradient on y and ``dtotal`` on t.  Returns (dx in total's type,
which is the gradient of x and of the residual, dweight [D] fp32).)";

}  // namespace

void init_layers(const py::dict& entries) {
  entry(entries, "selective_scan_forward_workspace_size", api.scan_workspace);
  entry(entries, "selective_scan_forward", api.scan);
  entry(entries, "selective_scan_backward_workspace_size", api.scan_backward_workspace);
  entry(entries, "selective_scan_backward", api.scan_backward);
  entry(entries, "selective_step", api.step);
  entry(entries, "causal_conv_forward", api.conv);
  entry(entries, "causal_conv_backward_workspace_size", api.conv_backward_workspace);
  entry(entries, "causal_conv_backward", api.conv_backward);
  entry(entries, "causal_conv_step", api.conv_step);
  entry(entries, "rms_norm_forward", api.norm);
  entry(entries, "rms_norm_quantize", api.norm_quantize);
  entry(entries, "rms_norm_backward_workspace_size", api.norm_backward_workspace);
  entry(entries, "rms_norm_backward", api.norm_backward);
}

void bind_layers(py::module_& mod) {
  using py::arg;
  const py::none none;
  py::options options;
  options.disable_function_signatures();
  mod.def("selective_scan_forward", &call_selective_scan, kScanDoc, arg("u"), arg("delta"), arg("A"), arg("B"), arg("C"),
          py::kw_only(), arg("skip") = none, arg("z") = none, arg("delta_bias") = none, arg("delta_softplus") = false,
          arg("h0") = none, arg("lengths") = none, arg("return_last") = false, arg("workspace") = none);
  mod.def("selective_scan_backward", &call_selective_scan_backward, kScanBackwardDoc, arg("u"), arg("delta"), arg("A"),
          arg("B"), arg("C"), arg("dy"), py::kw_only(), arg("skip") = none, arg("z") = none, arg("delta_bias") = none,
          arg("delta_softplus") = false, arg("h0") = none, arg("lengths") = none, arg("dh_last") = none,
          arg("workspace") = none);
  mod.def("selective_step", &call_selective_step, kStepDoc, arg("u"), arg("delta"), arg("A"), arg("B"), arg("C"),
          py::kw_only(), arg("skip") = none, arg("z") = none, arg("delta_bias") = none, arg("delta_softplus") = false,
          arg("h_prev") = none, arg("h_next") = none);
  mod.def("causal_conv_forward", &call_causal_conv, kConvDoc, arg("x"), arg("weight"), arg("bias") = none, py::kw_only(),
          arg("silu") = false, arg("state") = none, arg("lengths") = none, arg("return_last") = false);
  mod.def("causal_conv_backward", &call_causal_conv_backward, kConvBackwardDoc, arg("x"), arg("weight"), arg("dy"),
          arg("bias") = none, py::kw_only(), arg("silu") = false, arg("state") = none, arg("lengths") = none,
          arg("dlast") = none, arg("workspace") = none);
  mod.def("causal_conv_step", &call_causal_conv_step, kConvStepDoc, arg("x"), arg("weight"), arg("bias") = none,
          py::kw_only(), arg("silu") = false, arg("state") = none, arg("state_next") = none);
  mod.def("rms_norm_forward", &call_rms_norm, kNormDoc, arg("x"), arg("weight"), arg("residual") = none, py::kw_only(),
          arg("eps") = 1e-6);
  mod.def("rms_norm_quantize", &call_rms_norm_quantize, kNormQuantizeDoc, arg("x"), arg("weight"), arg("residual") = none,
          py::kw_only(), arg("eps") = 1e-6);
  mod.def("rms_norm_backward", &call_rms_norm_backward, kNormBackwardDoc, arg("total"), arg("weight"), arg("dy"),
          py::kw_only(), arg("dtotal") = none, arg("eps") = 1e-6, arg("workspace") = none);
}
