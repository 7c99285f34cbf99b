// Python binding of the 8-bit and AdamW calls, whose small calls take 3 us on
// the GPU: checks tensors, allocates outputs and workspaces through PyTorch's
// caching allocator and calls the C ABI on PyTorch's current stream, like the
// ctypes binding of the other calls, at a fraction of its time per call
// (a one-row matmul_i8 7.6 -> 4.0 to 4.9 us, an AdamW step over 49 tensors 32 -> 7.3
// to 8.9 us, by machine).
// The library's entry points come from the package (init), which has loaded
// the library; nothing is linked against it.

#include <torch/csrc/autograd/python_variable.h>

#include "binding_util.hpp"

namespace {

struct Api {
  decltype(&::quantize_rows) quantize_rows;
  decltype(&::quantize_columns) quantize_columns;
  decltype(&::matmul_i8) matmul_i8;
  decltype(&::mingru_step_i8_workspace_size) step_workspace;
  decltype(&::mingru_step_i8) step;
  decltype(&::mingru_forward_i8_workspace_size) forward_workspace;
  decltype(&::mingru_forward_i8) forward;
  decltype(&::adamw_step) adamw_step;
  decltype(&::adamw_step_each) adamw_step_each;
} api;

void init(const py::dict& entries, py::object error) {
  entry(entries, "scanrnn_last_error", last_error);
  entry(entries, "quantize_rows", api.quantize_rows);
  entry(entries, "quantize_columns", api.quantize_columns);
  entry(entries, "matmul_i8", api.matmul_i8);
  entry(entries, "mingru_step_i8_workspace_size", api.step_workspace);
  entry(entries, "mingru_step_i8", api.step);
  entry(entries, "mingru_forward_i8_workspace_size", api.forward_workspace);
  entry(entries, "mingru_forward_i8", api.forward);
  entry(entries, "adamw_step", api.adamw_step);
  entry(entries, "adamw_step_each", api.adamw_step_each);
  error_class = error.release().ptr();
  init_layers(entries);
}

// ------------------------------------------------------------------- codes

struct CodeOut {
  Tensor q, scale;
};
CodeOut code_out(const MaybeTensor& q, const MaybeTensor& scale, int64_t n, int64_t K, const Tensor& like) {
  const int64_t width = stored_width(K);
  if (q) in_place(*q, "q", at::kChar, {n, width}, like);
  if (scale) in_place(*scale, "scale", at::kFloat, {n}, like);
  return {q ? *q : make(like, {n, width}, at::kChar), scale ? *scale : make(like, {n}, at::kFloat)};
}

std::pair<Tensor, Tensor> call_quantize_rows(const Tensor& x, const MaybeTensor& q, const MaybeTensor& scale) {
  const Rows r = rows_of(x, "x", 0);
  CodeOut out = code_out(q, scale, r.n, r.width, x);
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.quantize_rows(r.n, r.width, data(r.t), r.stride, r.type, data<int8_t>(out.q), data<float>(out.scale),
                           stream_of(x));
  }
  check("quantize_rows", st);
  written(q);
  written(scale);
  if (q || scale || x.dim() == 2) return {out.q, out.scale};
  std::vector<int64_t> shape(x.sizes().begin(), x.sizes().end() - 1);
  Tensor s = out.scale.view(shape);
  shape.push_back(out.q.size(1));
  return {out.q.view(shape), s};
}

std::pair<Tensor, Tensor> call_quantize_columns(const Tensor& W, const MaybeTensor& q, const MaybeTensor& scale) {
  const Rows r = rows_of(W, "W", 2);
  const int64_t K = r.n, N = r.width;
  CodeOut out = code_out(q, scale, N, K, W);
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.quantize_columns(K, N, data(r.t), r.stride, r.type, data<int8_t>(out.q), data<float>(out.scale),
                              stream_of(W));
  }
  check("quantize_columns", st);
  written(q);
  written(scale);
  return {out.q, out.scale};
}

Tensor call_matmul_i8(const Tensor& a, const Tensor& a_scale, const Tensor& b, const Tensor& b_scale,
                 at::ScalarType out_dtype, const MaybeTensor& out) {
  const Rows ra = codes_of(a, "a", 0), rb = codes_of(b, "b", 2);
  if (ra.width != rb.width)
    bad_value("a and b must have rows of the same width (got " + std::to_string(ra.width) + " and " +
              std::to_string(rb.width) + ")");
  same_device(b, "b", a);
  const Tensor sa = scales_of(a_scale, "a_scale", ra.n, a), sb = scales_of(b_scale, "b_scale", rb.n, a);
  std::vector<int64_t> shape(a.sizes().begin(), a.sizes().end() - 1);
  shape.push_back(rb.n);
  Tensor y;
  if (out) {
    float_type(*out, "out");
    in_place(*out, "out", out->scalar_type(), shape, a);
    y = *out;
  } else {
    if (out_dtype != at::kFloat && out_dtype != at::kBFloat16)
      bad_type(std::string("out_dtype must be float32 or bfloat16 (got ") + at::toString(out_dtype) + ")");
    y = make(a, shape, out_dtype);
  }
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.matmul_i8(ra.n, rb.n, ra.width, data<int8_t>(ra.t), ra.stride, data<float>(sa), data<int8_t>(rb.t),
                       rb.stride, data<float>(sb), data(y), rb.n, y.scalar_type() == at::kFloat ? SR_F32 : SR_BF16,
                       stream_of(a));
  }
  check("matmul_i8", st);
  written(out);
  return y;
}

// ------------------------------------------------------------ minGRU modes

struct Weights {
  Tensor W_in, W_in_scale;
  MaybeTensor W_out, W_out_scale;
  int64_t D_h, D_out;
};
Tensor weight_codes(const Tensor& t, const char* name, int64_t width, const Tensor& like) {
  const Rows r = codes_of(t, name, 2);
  if (r.width != width)
    bad_value(std::string(name) + " must have rows of " + std::to_string(width) + " codes (got shape " +
              text(t.sizes()) + ")");
  same_device(t, name, like);
  return r.stride == width ? r.t : r.t.contiguous();
}
Weights weights_of(int64_t D_in, const Tensor& W_in, const Tensor& W_in_scale, const MaybeTensor& W_out,
                   const MaybeTensor& W_out_scale, const Tensor& like) {
  Weights w;
  w.W_in = weight_codes(W_in, "W_in", stored_width(D_in), like);
  if (W_in.size(0) % 2) bad_value("W_in must have 2*D_h rows (got " + std::to_string(W_in.size(0)) + ")");
  w.W_in_scale = scales_of(W_in_scale, "W_in_scale", W_in.size(0), like);
  w.D_h = w.D_out = W_in.size(0) / 2;
  if (W_out.has_value() != W_out_scale.has_value()) bad_value("W_out and W_out_scale go together");
  if (W_out) {
    w.W_out = weight_codes(*W_out, "W_out", stored_width(w.D_h), like);
    w.D_out = W_out->size(0);
    w.W_out_scale = scales_of(*W_out_scale, "W_out_scale", w.D_out, like);
  }
  return w;
}

struct DecayArgs {
  MaybeTensor rate, gap, saturated;
};
DecayArgs decay_of(const MaybeTensor& rate, const MaybeTensor& gap, const MaybeTensor& saturated, int64_t D_h,
                   at::IntArrayRef gap_shape, const Tensor& like) {
  DecayArgs d;
  if (!rate) {
    if (gap || saturated) bad_value("delta_t and saturated need decay_rate");
    return d;
  }
  if (!gap) bad_value("decay_rate and delta_t go together");
  has_type(*rate, "decay_rate", at::kFloat);
  has_shape(*rate, "decay_rate", {D_h});
  same_device(*rate, "decay_rate", like);
  has_type(*gap, "delta_t", at::kFloat);
  has_shape(*gap, "delta_t", gap_shape);
  same_device(*gap, "delta_t", like);
  d.rate = rate->contiguous();
  d.gap = gap->contiguous();
  if (saturated) {
    has_type(*saturated, "saturated", at::kInt);
    if (saturated->numel() < 1 || !saturated->is_contiguous())
      bad_value("saturated must be a contiguous int32 tensor of at least one element");
    same_device(*saturated, "saturated", like);
    d.saturated = saturated;
  }
  return d;
}

std::pair<Tensor, Tensor> call_mingru_step_i8(const Tensor& x_t, const Tensor& W_in, const Tensor& W_in_scale,
                                         const MaybeTensor& W_out, const MaybeTensor& W_out_scale,
                                         const MaybeTensor& h_prev, const MaybeTensor& h_next,
                                         const MaybeTensor& workspace, const MaybeTensor& decay_rate,
                                         const MaybeTensor& delta_t, bool log1p_delta, const MaybeTensor& saturated) {
  const sr_dtype type = float_type(x_t, "x_t");
  if (x_t.dim() != 2) bad_value("x_t must have 2 dims (got shape " + text(x_t.sizes()) + ")");
  const Tensor x = x_t.contiguous();
  const int64_t B = x.size(0), D_in = x.size(1);
  const Weights w = weights_of(D_in, W_in, W_in_scale, W_out, W_out_scale, x);
  if (h_prev) in_place(*h_prev, "h_prev", at::kFloat, {B, w.D_h}, x);
  if (h_next) in_place(*h_next, "h_next", at::kFloat, {B, w.D_h}, x);
  const DecayArgs d = decay_of(decay_rate, delta_t, saturated, w.D_h, {B}, x);
  const Tensor h = h_next ? *h_next : make(x, {B, w.D_h}, at::kFloat);
  MaybeTensor y;
  if (w.W_out) y = make(x, {B, w.D_out}, x.scalar_type());
  const Tensor ws = workspace_of(workspace, api.step_workspace(B, D_in, w.D_h, w.D_out), x);
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.step(B, D_in, w.D_h, w.D_out, data(x), type, operand<int8_t>(w.W_in), operand<float>(w.W_in_scale),
                  operand<int8_t>(w.W_out), operand<float>(w.W_out_scale), data<float>(d.rate), data<float>(d.gap),
                  log1p_delta, data<uint32_t>(d.saturated), data<float>(h_prev), data<float>(h), data(y),
                  ws.data_ptr(), size_t(ws.numel()), stream_of(x));
  }
  check("mingru_step_i8", st);
  written(h_next);
  written(saturated);
  return {y ? *y : h, h};
}

py::object call_mingru_forward_i8(const Tensor& x_in, const Tensor& W_in, const Tensor& W_in_scale,
                             const MaybeTensor& W_out, const MaybeTensor& W_out_scale, const MaybeTensor& h0_in,
                             bool return_last, const MaybeTensor& workspace, const MaybeTensor& decay_rate,
                             const MaybeTensor& delta_t, bool log1p_delta, const MaybeTensor& saturated) {
  const sr_dtype type = float_type(x_in, "x");
  if (x_in.dim() != 3) bad_value("x must have 3 dims (got shape " + text(x_in.sizes()) + ")");
  const Tensor x = x_in.contiguous();
  const int64_t B = x.size(0), T = x.size(1), D_in = x.size(2);
  const Weights w = weights_of(D_in, W_in, W_in_scale, W_out, W_out_scale, x);
  MaybeTensor h0;
  if (h0_in) {
    h0 = h0_in->contiguous();
    in_place(*h0, "h0", at::kFloat, {B, w.D_h}, x);
  }
  const DecayArgs d = decay_of(decay_rate, delta_t, saturated, w.D_h, {B, T}, x);
  const Tensor y = make(x, {B, T, w.D_out}, w.W_out ? x.scalar_type() : at::kFloat);
  MaybeTensor last;
  if (return_last) last = make(x, {B, w.D_h}, at::kFloat);
  const Tensor ws =
      workspace_of(workspace, api.forward_workspace(B, T, D_in, w.D_h, w.D_out, type, w.W_out.has_value()), x);
  sr_status st;
  {
    py::gil_scoped_release release;
    st = api.forward(B, T, D_in, w.D_h, w.D_out, data(x), type, operand<int8_t>(w.W_in), operand<float>(w.W_in_scale),
                     operand<int8_t>(w.W_out), operand<float>(w.W_out_scale), data<float>(d.rate), data<float>(d.gap),
                     log1p_delta, data<uint32_t>(d.saturated), data<float>(h0), data(y), data<float>(last),
                     ws.data_ptr(), size_t(ws.numel()), stream_of(x));
  }
  check("mingru_forward_i8", st);
  written(saturated);
  if (!return_last) return py::cast(y);
  return py::make_tuple(y, *last);
}

// ------------------------------------------------------------------- AdamW

// The tensors of a sequence; an undefined one for None, where that is allowed.
std::vector<Tensor> tensors_of(const py::handle& sequence, const char* name, bool or_none) {
  py::object fast = py::reinterpret_steal<py::object>(PySequence_Fast(sequence.ptr(), "a sequence of tensors is wanted"));
  if (!fast) throw py::error_already_set();
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast.ptr());
  PyObject** items = PySequence_Fast_ITEMS(fast.ptr());
  std::vector<Tensor> out(static_cast<size_t>(n));
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (THPVariable_Check(items[i]))
      out[size_t(i)] = THPVariable_Unpack(items[i]);
    else if (!or_none || items[i] != Py_None)
      bad_type(std::string(name) + "[" + std::to_string(i) + "] must be a torch.Tensor");
  }
  return out;
}

int64_t integer(const py::handle& x) {
  const py::object index = py::reinterpret_steal<py::object>(PyNumber_Index(x.ptr()));
  if (!index) throw py::error_already_set();
  const int64_t n = PyLong_AsLongLong(index.ptr());
  if (n == -1 && PyErr_Occurred()) throw py::error_already_set();
  return n;
}

// The step numbers of n tensors.
std::vector<int64_t> steps_of(const py::object& step, size_t n) {
  const py::object fast =
      py::reinterpret_steal<py::object>(PySequence_Fast(step.ptr(), "step must be an integer or a sequence of them"));
  if (!fast) throw py::error_already_set();
  if (size_t(PySequence_Fast_GET_SIZE(fast.ptr())) != n)
    bad_value(std::to_string(n) + " params but " + std::to_string(PySequence_Fast_GET_SIZE(fast.ptr())) + " steps");
  std::vector<int64_t> out(n);
  for (size_t i = 0; i < n; ++i) out[i] = integer(PySequence_Fast_GET_ITEM(fast.ptr(), Py_ssize_t(i)));
  return out;
}

int64_t call_adamw_step(const py::object& params, const py::object& grads, const Tensor& m, const Tensor& v,
                        const py::object& step, const MaybeTensor& m_scale, const MaybeTensor& v_scale, double lr,
                        std::pair<double, double> betas, double eps, double weight_decay,
                        const MaybeTensor& grad_scale) {
  const std::vector<Tensor> ps = tensors_of(params, "params", false), gs = tensors_of(grads, "grads", true);
  if (ps.size() != gs.size())
    bad_value(std::to_string(ps.size()) + " params but " + std::to_string(gs.size()) + " grads");
  const bool one = PyIndex_Check(step.ptr());
  const int64_t number = one ? integer(step) : 0;
  const std::vector<int64_t> steps = one ? std::vector<int64_t>() : steps_of(step, ps.size());
  if (ps.empty()) return 0;
  std::vector<sr_adamw_tensor> table(ps.size());
  for (size_t i = 0; i < ps.size(); ++i) {
    const Tensor &p = ps[i], &g = gs[i];
    sr_adamw_tensor& t = table[i];
    const auto usable = [&](const Tensor& x) {
      return x.device() == ps[0].device() && x.is_cuda() && x.is_contiguous() &&
             (x.scalar_type() == at::kFloat || x.scalar_type() == at::kBFloat16);
    };
    if (!usable(p))
      bad_value("params[" + std::to_string(i) + "] must be a contiguous float32 or bfloat16 tensor on one GPU");
    if (g.defined() && !(usable(g) && g.sizes() == p.sizes()))
      bad_value("grads[" + std::to_string(i) + "] must be a contiguous float32 or bfloat16 tensor of shape " +
                text(p.sizes()) + " on " + p.device().str());
    t.param = p.data_ptr();
    t.grad = g.defined() ? g.data_ptr() : nullptr;
    t.n = p.numel();
    t.param_dtype = p.scalar_type() == at::kBFloat16 ? SR_BF16 : SR_F32;
    t.grad_dtype = g.defined() && g.scalar_type() == at::kBFloat16 ? SR_BF16 : SR_F32;
  }
  const bool eight = m_scale || v_scale;
  if (eight && !(m_scale && v_scale)) bad_value("m_scale and v_scale go together");
  const int64_t n = m.numel();
  const at::ScalarType type = eight ? at::kFloat8_e4m3fn : at::kFloat;
  in_place(m, "m", type, {n}, ps[0]);
  in_place(v, "v", type, {n}, ps[0]);
  if (eight) {
    in_place(*m_scale, "m_scale", at::kFloat, {n / 256}, ps[0]);
    in_place(*v_scale, "v_scale", at::kFloat, {n / 256}, ps[0]);
  }
  MaybeTensor gs_value;
  if (grad_scale) gs_value = scales_of(*grad_scale, "grad_scale", 1, ps[0]);
  sr_status st;
  {
    py::gil_scoped_release release;
    const auto call = [&](auto* fn, auto which) {
      return fn(int64_t(table.size()), table.data(), data(m), data(v), data<float>(m_scale), data<float>(v_scale),
                eight ? 8 : 32, n, which, lr, betas.first, betas.second, eps, weight_decay, data<float>(gs_value),
                stream_of(ps[0]));
    };
    st = one ? call(api.adamw_step, number) : call(api.adamw_step_each, steps.data());
  }
  check("adamw_step", st);
  int64_t moved = 0;
  for (size_t i = 0; i < ps.size(); ++i) {
    if (!gs[i].defined()) continue;
    written(ps[i]);
    ++moved;
  }
  written(m);
  written(v);
  written(m_scale);
  written(v_scale);
  return moved;
}

constexpr const char* kRowsDoc = R"(quantize_rows(x, q=None, scale=None)

Symmetric 8-bit codes of the rows (last dimension) of ``x`` [.., K], fp32 or
bf16, with a scale each: scale = max|x| / 127, q = rint(x / scale).

Returns (q [.., quantized_row_bytes(K)] int8, zeros behind the K codes, scale
[..] fp32).  A row of zeros has scale 0; a row with a NaN or an infinity has
scale NaN and codes 0.  ``q`` [rows, ..] and ``scale`` [rows] may be given to
avoid the allocations.)";
constexpr const char* kColumnsDoc = R"(quantize_columns(W, q=None, scale=None)

8-bit codes of the columns of a weight ``W`` [K, N] (an output channel each),
laid out for matmul_i8: (q [N, quantized_row_bytes(K)] int8, scale [N] fp32), as
quantize_rows of its transpose.)";
constexpr const char* kMatmulDoc = R"(matmul_i8(a, a_scale, b, b_scale, out_dtype=torch.float32, out=None)

y[.., n] = (sum_k a[.., k] b[n, k]) (a_scale[..] b_scale[n]): the product of
codes ``a`` [.., K] (quantize_rows) and ``b`` [N, K] (quantize_columns), summed
exactly in 32-bit integers.  K is the stored width, a multiple of 128.  Returns y
[.., N] in ``out_dtype`` (float32 or bfloat16).)";
constexpr const char* kStepDoc =
    R"(mingru_step_i8(x_t, W_in, W_in_scale, W_out=None, W_out_scale=None, h_prev=None, h_next=None, workspace=None,
               *, decay_rate=None, delta_t=None, log1p_delta=False, saturated=None)

``mingru_step`` on 8-bit weights: x_t [B,D_in] fp32 or bf16 -> (y_t [B,D_out] in
x_t's type, h_t [B,D_h] fp32).

``W_in`` and ``W_out`` are the codes of the layer's weights with their scales
(quantize_columns); x_t and the new state are quantised row by row inside the
call.  Without ``W_out`` the output is the new state (the same tensor is returned
twice).  ``h_next`` may be ``h_prev`` (a step in place); it must not share memory with
another part of it, nor with x_t.  ``decay_rate`` [D_h] with ``delta_t`` [B]: time decay as in
``mingru_step_decayed``.)";
constexpr const char* kForwardDoc =
    R"(mingru_forward_i8(x, W_in, W_in_scale, W_out=None, W_out_scale=None, h0=None, return_last=False, workspace=None,
                  *, decay_rate=None, delta_t=None, log1p_delta=False, saturated=None)

``mingru_forward`` on 8-bit weights: x [B,T,D_in] fp32 or bf16 -> y [B,T,D_out]
in x's type (without ``W_out`` the states, in fp32), and h_T [B,D_h] fp32 when
``return_last``.  Arguments as in ``mingru_step_i8``; the gate logits and
candidates reach the scan in x's type.)";
constexpr const char* kAdamWDoc =
    R"(adamw_step(params, grads, m, v, *, step, m_scale=None, v_scale=None, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
           weight_decay=1e-2, grad_scale=None)

One AdamW step over many tensors, in place on ``params`` and the states.
Returns how many of them had a gradient.

``params`` and ``grads``: lists of contiguous GPU tensors of the same shapes,
fp32 or bf16 each; a gradient may be None (that tensor is left as it is).  A
parameter is given once: tensors that share memory are refused.
``step`` counts from 1: a number for all of them, or a list of one for each.
``m`` and ``v`` hold the states of all tensors one after another, each tensor's
span rounded up to 256 elements (``adamw_state_elements``):
fp32 without scales, or float8_e4m3fn codes (of m and
of sqrt(v)) with one fp32 scale for each 256 elements in ``m_scale`` and
``v_scale``.  Zeros are the states before the first step.  ``grad_scale``: an fp32
GPU scalar multiplied onto every gradient.

Limit of the float8 states: codes of sqrt(v) are 6 to 12 percent apart and one
step moves it by less, so an element follows the largest of its 256, which is held
exactly.  While the gradients of a block keep their proportions, sqrt(v) stays
within about 0.7 to 1.7 of its fp32 value; an element whose gradients shrink
against the rest of its block keeps its old one, and one whose gradients grow falls
behind by up to about 8 times (beta2 = 0.999; 3 times with 0.99): its steps are too
small, or too large, by that factor.  Where that matters, use fp32 states.)";

}  // namespace

PYBIND11_MODULE(_binding, mod) {
  using py::arg;
  const py::none none;
  py::options options;
  options.disable_function_signatures();
  mod.def("init", &init);
  bind_layers(mod);
  mod.def("quantize_rows", &call_quantize_rows, kRowsDoc, arg("x"), arg("q") = none, arg("scale") = none);
  mod.def("quantize_columns", &call_quantize_columns, kColumnsDoc, arg("W"), arg("q") = none, arg("scale") = none);
  mod.def("matmul_i8", &call_matmul_i8, kMatmulDoc, arg("a"), arg("a_scale"), arg("b"), arg("b_scale"),
          arg("out_dtype") = at::kFloat, arg("out") = none);
  mod.def("mingru_step_i8", &call_mingru_step_i8, kStepDoc, arg("x_t"), arg("W_in"), arg("W_in_scale"),
          arg("W_out") = none, arg("W_out_scale") = none, arg("h_prev") = none, arg("h_next") = none,
          arg("workspace") = none, py::kw_only(), arg("decay_rate") = none, arg("delta_t") = none,
          arg("log1p_delta") = false, arg("saturated") = none);
  mod.def("mingru_forward_i8", &call_mingru_forward_i8, kForwardDoc, arg("x"), arg("W_in"), arg("W_in_scale"),
          arg("W_out") = none, arg("W_out_scale") = none, arg("h0") = none, arg("return_last") = false,
          arg("workspace") = none, py::kw_only(), arg("decay_rate") = none, arg("delta_t") = none,
          arg("log1p_delta") = false, arg("saturated") = none);
  mod.def("adamw_step", &call_adamw_step, kAdamWDoc, arg("params"), arg("grads"), arg("m"), arg("v"), py::kw_only(),
          arg("step"), arg("m_scale") = none, arg("v_scale") = none, arg("lr") = 1e-3,
          arg("betas") = std::make_pair(0.9, 0.999), arg("eps") = 1e-8, arg("weight_decay") = 1e-2,
          arg("grad_scale") = none);
}
