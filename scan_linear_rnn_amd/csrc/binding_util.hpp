// What the binding's sources share: checks of tensors, outputs and workspaces
// from PyTorch's caching allocator, its current stream, errors.
#pragma once

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <vector>

#include "scanrnn.h"

namespace py = pybind11;
using at::Tensor;
using MaybeTensor = std::optional<Tensor>;

// binding_layers.cpp: the selective scan, the convolution and the norm.
void init_layers(const py::dict& entries);
void bind_layers(py::module_& mod);

inline PyObject* error_class = nullptr;  // ScanRNNError(function, status, message)
inline decltype(&::scanrnn_last_error) last_error = nullptr;

template <class F>
void entry(const py::dict& entries, const char* name, F& fn) {
  fn = reinterpret_cast<F>(entries[name].cast<uintptr_t>());
}

// ------------------------------------------------------------------ checks

[[noreturn]] inline void bad_value(const std::string& what) { throw py::value_error(what); }
[[noreturn]] inline void bad_type(const std::string& what) { throw py::type_error(what); }

inline std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}

inline void check(const char* fn, sr_status st) {
  if (st == SR_OK) return;
  py::object error = py::reinterpret_borrow<py::object>(error_class)(fn, int(st), std::string(last_error()));
  PyErr_SetObject(error_class, error.ptr());
  throw py::error_already_set();
}

inline void on_gpu(const Tensor& t, const std::string& name) {
  if (!t.defined() || !t.is_cuda())
    bad_value(name + " must be a GPU tensor (got " + (t.defined() ? t.device().str() : "none") + ")");
}
inline void has_type(const Tensor& t, const std::string& name, at::ScalarType want) {
  on_gpu(t, name);
  if (t.scalar_type() != want)
    bad_type(name + " must be " + at::toString(want) + " (got " + at::toString(t.scalar_type()) + ")");
}
inline sr_dtype float_type(const Tensor& t, const std::string& name) {
  on_gpu(t, name);
  if (t.scalar_type() == at::kFloat) return SR_F32;
  if (t.scalar_type() == at::kBFloat16) return SR_BF16;
  bad_type(name + " must be float32 or bfloat16 (got " + at::toString(t.scalar_type()) + ")");
}
inline void same_device(const Tensor& t, const std::string& name, const Tensor& like) {
  if (t.device() != like.device())
    bad_value(name + " must be on " + like.device().str() + " (got " + t.device().str() + ")");
}
inline void has_shape(const Tensor& t, const std::string& name, at::IntArrayRef shape) {
  if (t.sizes() != shape) bad_value(name + " must have shape " + text(shape) + " (got " + text(t.sizes()) + ")");
}
// A tensor that is written or carried: contiguous as it is.
inline void in_place(const Tensor& t, const std::string& name, at::ScalarType type, at::IntArrayRef shape, const Tensor& like) {
  has_type(t, name, type);
  has_shape(t, name, shape);
  if (!t.is_contiguous()) bad_value(name + " must be contiguous");
  same_device(t, name, like);
}

template <class T = void>
T* data(const Tensor& t) { return t.numel() ? static_cast<T*>(t.data_ptr()) : nullptr; }
template <class T = void>
T* data(const MaybeTensor& t) { return t ? data<T>(*t) : nullptr; }
// An optional weight that is present but has no elements (no input features,
// no state) still has to read as present: an address that is never followed.
template <class T>
const T* operand(const MaybeTensor& t) {
  if (!t) return nullptr;
  return t->numel() ? static_cast<const T*>(t->data_ptr()) : reinterpret_cast<const T*>(uintptr_t(4096));
}

// After a call has written them, tensors of the caller's count a version up, as
// PyTorch's own in-place operations do: a backward pass that saved one of them
// before is then refused.  (Tensors made in inference mode have no version.)
inline void written(const Tensor& t) {
  if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
inline void written(const MaybeTensor& t) {
  if (t) written(*t);
}

inline void* stream_of(const Tensor& t) {
  return c10::hip::getCurrentHIPStream(t.device().index()).stream();
}

inline Tensor make(const Tensor& like, at::IntArrayRef shape, at::ScalarType type) {
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

inline int64_t stored_width(int64_t K) { return (K + 127) / 128 * 128; }

// fp32 or bf16 as rows of its last dimension: a view when it can be one.
struct Rows {
  Tensor t;
  int64_t n, width, stride;
  sr_dtype type;
};
inline Rows rows_of(const Tensor& t, const char* name, int64_t dims) {
  Rows r;
  r.type = float_type(t, name);
  if (dims ? t.dim() != dims : t.dim() < 1)
    bad_value(std::string(name) + " must have " + (dims ? std::to_string(dims) : "at least one") +
              " dims (got shape " + text(t.sizes()) + ")");
  r.width = t.size(-1);
  r.n = 1;
  for (int64_t i = 0; i + 1 < t.dim(); ++i) r.n *= t.size(i);
  if (t.dim() == 2 && r.n > 1 && t.stride(1) == 1 && t.stride(0) >= r.width) {
    r.t = t;
    r.stride = t.stride(0);
  } else {
    r.t = t.contiguous();
    r.stride = r.width;
  }
  return r;
}

// Codes [.., K] as rows.
inline Rows codes_of(const Tensor& t, const char* name, int64_t dims) {
  has_type(t, name, at::kChar);
  if (dims ? t.dim() != dims : t.dim() < 2)
    bad_value(std::string(name) + " must have " + (dims ? std::to_string(dims) : "at least 2") +
              " dims (got shape " + text(t.sizes()) + ")");
  Rows r;
  r.width = t.size(-1);
  if (r.width % 128)
    bad_value(std::string(name) + " must have rows of a multiple of 128 codes, zeros behind the data (got " +
              std::to_string(r.width) + ")");
  r.n = 1;
  for (int64_t i = 0; i + 1 < t.dim(); ++i) r.n *= t.size(i);
  const auto aligned = [](const Tensor& x) { return reinterpret_cast<uintptr_t>(x.data_ptr()) % 16 == 0; };
  if (t.dim() == 2 && r.n > 1 && t.stride(1) == 1 && t.stride(0) >= r.width && t.stride(0) % 16 == 0 && aligned(t)) {
    r.t = t;
    r.stride = t.stride(0);
  } else {
    r.t = t.contiguous();
    if (!aligned(r.t)) r.t = r.t.clone();
    r.stride = r.width;
  }
  return r;
}

inline Tensor scales_of(const Tensor& t, const std::string& name, int64_t n, const Tensor& like) {
  has_type(t, name, at::kFloat);
  if (t.numel() != n)
    bad_value(name + " must have " + std::to_string(n) + " elements (got shape " + text(t.sizes()) + ")");
  same_device(t, name, like);
  return t.contiguous();
}

inline Tensor workspace_of(const MaybeTensor& workspace, size_t bytes, const Tensor& like) {
  if (!workspace) return make(like, {int64_t(bytes ? bytes : 1)}, at::kByte);
  if (workspace->scalar_type() != at::kByte) bad_type("workspace must be a torch.uint8 tensor");
  if (workspace->device() != like.device() || !workspace->is_contiguous())
    bad_value("workspace must be a contiguous tensor on " + like.device().str());
  if (size_t(workspace->numel()) < bytes)
    bad_value("workspace has " + std::to_string(workspace->numel()) + " bytes, " + std::to_string(bytes) + " needed");
  return *workspace;
}
