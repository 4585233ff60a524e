// What the extensions that call the library on torch tensors share: an
// operator's plan, the checks of a call's tensors, and refusals as exceptions.
#pragma once

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>

#include <optional>
#include <string>

#include "../../include/kfac_objectives.h"

namespace {

// An operator's workspace, device (-1: not a GPU) and constant fields.
struct Plan {
  void* ws;
  size_t ws_bytes;
  PyObject* ws_tensor;  // the tensor that holds the workspace, kept by the operator; NULL: none
  void* home;           // the stream it was allocated on
  const char* name;
  int32_t device;
  int32_t dtype;
};
PyObject* error_class = nullptr;

struct Refused {
  int status;
  std::string what;
};

class Call {
 public:
  explicit Call(const Plan& plan) : plan_(plan) {}

  [[noreturn]] void refuse(const std::string& what, int status = KFAC_ERR_ARG) const {
    throw Refused{status, std::string(plan_.name) + ": " + what};
  }

  at::ScalarType dtype() const { return plan_.dtype == KFAC_BF16 ? at::kBFloat16 : at::kFloat; }

  const at::Tensor& tensor(PyObject* o, const char* name) const {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
  }

  // A tensor that a derivative may be taken through.  The backward passes are there, but no operator carries a
  // forward-mode tangent on (without this its result would have none: a derivative of zero).
  const at::Tensor& differentiable(PyObject* o, const char* name) const {
    const at::Tensor& t = tensor(o, name);
    if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined())
      refuse(std::string(name) + " has a forward-mode tangent, and the operator no forward-mode derivative", KFAC_ERR_UNSUPPORTED);
    return t;
  }

  bool placed(const at::Tensor& t) const {
    if (t.layout() != at::kStrided) return false;
    return plan_.device < 0 ? t.is_cpu() : t.is_cuda() && t.get_device() == plan_.device;
  }
  std::string place() const { return plan_.device < 0 ? "the CPU" : "cuda:" + std::to_string(plan_.device); }

  // [rows, cols] of a dtype (KFAC_F32, KFAC_BF16) with adjacent columns; its row stride goes to `ld`.
  void* matrix_of(const at::Tensor& t, const char* name, int32_t want, int64_t rows, int64_t cols, int64_t* ld) const {
    if (t.scalar_type() != (want == KFAC_BF16 ? at::kBFloat16 : at::kFloat))
      refuse(std::string(name) + " must be " + (want == KFAC_BF16 ? "bfloat16" : "float32"), KFAC_ERR_DTYPE);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || !placed(t))
      refuse(std::string(name) + " must be [" + std::to_string(rows) + ", " + std::to_string(cols) + "] on " + place());
    *ld = rows < 2 ? cols : t.stride(0);
    if ((t.stride(1) != 1 && cols > 1) || *ld < cols)
      refuse(std::string(name) + " must have adjacent columns and rows that do not overlap");
    return t.data_ptr();
  }
  // The same of the operator's own dtype.
  void* matrix(const at::Tensor& t, const char* name, int64_t rows, int64_t cols, int64_t* ld) const {
    return matrix_of(t, name, plan_.dtype, rows, cols, ld);
  }

  // n contiguous values of one dtype.
  void* vector(PyObject* o, const char* name, int64_t n, at::ScalarType want) const {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != want) refuse(std::string(name) + " must be " + c10::toString(want), KFAC_ERR_DTYPE);
    if (t.numel() != n || !placed(t) || !t.is_contiguous())
      refuse(std::string(name) + " must be " + std::to_string(n) + " contiguous values on " + place());
    return t.data_ptr();
  }
  float* floats(PyObject* o, const char* name, int64_t n) const {
    return o == Py_None ? nullptr : static_cast<float*>(vector(o, name, n, at::kFloat));
  }

  // Contiguous int32 or int64 indices [n] or [n, k]; their type goes to `type`.
  void* indices(PyObject* o, const char* name, int64_t n, int64_t k, int32_t* type) const {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong)
      refuse(std::string(name) + " must be int32 or int64", KFAC_ERR_DTYPE);
    const bool fits = k < 0 ? t.dim() == 1 && t.size(0) == n : t.dim() == 2 && t.size(0) == n && t.size(1) == k;
    if (!fits || !placed(t) || !t.is_contiguous())
      refuse(std::string(name) + " must be [" + std::to_string(n) + (k < 0 ? "" : ", " + std::to_string(k)) +
             "], contiguous, on " + place());
    *type = t.scalar_type() == at::kLong ? KFAC_I64 : KFAC_I32;
    return t.data_ptr();
  }

  // The GPU's current stream; from here on everything is allocated and runs there.
  void* enter() {
    if (plan_.device < 0) refuse("the operators run on a GPU only", KFAC_ERR_UNSUPPORTED);
    guard_.emplace(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(plan_.device)));
    options_ = at::TensorOptions().device(c10::kCUDA, static_cast<c10::DeviceIndex>(plan_.device)).dtype(at::kFloat);
    const auto stream = c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(static_cast<c10::DeviceIndex>(plan_.device));
    // an operator may go while its call still runs elsewhere: the allocator then waits for that stream
    if (plan_.ws_tensor && stream.stream() != plan_.home) THPVariable_Unpack(plan_.ws_tensor).record_stream(stream.unwrap());
    return stream.stream();
  }
  at::Tensor make(int64_t n, at::ScalarType type = at::kFloat) const { return at::empty({n}, options_.dtype(type)); }

  // Contiguous, of KFAC_F32 or KFAC_BF16.
  at::Tensor make_like(at::IntArrayRef sizes, int32_t dtype) const {
    return at::empty(sizes, options_.dtype(dtype == KFAC_BF16 ? at::kBFloat16 : at::kFloat));
  }
  at::Tensor make_matrix(int64_t rows, int64_t cols, int32_t dtype) const { return make_like({rows, cols}, dtype); }

  // A gradient for logits of row stride ld: every row at the same place within
  // 16 bytes as the logits' row, at the least width.
  at::Tensor make_rows(int64_t rows, int64_t cols, int64_t ld, int64_t* out_ld) const {
    const int64_t per = plan_.dtype == KFAC_BF16 ? 8 : 4;
    *out_ld = cols + (ld - cols) % per;
    return at::empty_strided({rows, cols}, {*out_ld, 1}, options_.dtype(dtype()));
  }

 private:
  const Plan& plan_;
  std::optional<c10::DeviceGuard> guard_;
  at::TensorOptions options_;
};

// Runs `body`, which returns the outputs; refusals and failures become exceptions.
template <typename F>
PyObject* guarded(F&& body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const Refused& r) {
    PyObject* e = PyObject_CallFunction(error_class, "is", r.status, r.what.c_str());
    if (e) {
      PyErr_SetObject(error_class, e);
      Py_DECREF(e);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

void done(kfac_status_t s, const char* fn) {
  if (s != KFAC_OK) throw Refused{s, fn};
}

template <typename P>
const P* plan_of(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw Refused{KFAC_ERR_ARG, "wrong number of arguments"};
  const P* p = static_cast<const P*>(PyLong_AsVoidPtr(args[0]));
  if (!p) throw Refused{KFAC_ERR_ARG, "no plan"};
  return p;
}

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(t));
  return out;
}

// The caller's output tensor has been written: operations that saved it for a
// backward pass find out, as after torch's own writes in place.  (A tensor of
// inference mode cannot be saved, and counts no writes.)
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

template <typename F>
PyCFunction method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

}  // namespace
