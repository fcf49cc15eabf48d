// bind_common.hpp -- what the binding's files share: checks of tensors, outputs
// and scratch, errors, and refusals of what would go past torch's dispatcher.

#pragma once

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/Allocator.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/saved_variable.h>
#include <torch/csrc/autograd/variable.h>
#include <torch/csrc/jit/frontend/tracer.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <vector>

#include "ssim_train_amd.h"

namespace py = pybind11;

namespace ssim_bind {

using at::Tensor;

inline std::string text(int code) {
  return std::string(ssim_train_strerror(code)) + " (code " + std::to_string(code) + ")";
}

// Python callers get the package's TrainError
inline void raise(int code, const char* where) {
  py::object type = py::module_::import("ssim_loss_amd.train").attr("TrainError");
  py::object error = type(code, where);
  PyErr_SetObject(type.ptr(), error.ptr());
  throw py::error_already_set();
}

inline std::string at_index(const char* name, Py_ssize_t k) {
  return k < 0 ? std::string(name) : std::string(name) + "[" + std::to_string(k) + "]";
}

inline int dtype_code(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return SSIM_DTYPE_F32;
    case at::kHalf: return SSIM_DTYPE_F16;
    case at::kBFloat16: return SSIM_DTYPE_BF16;
    default: return -1;
  }
}

// a GPU tensor of one of the three types, contiguous or (dense) without gaps in
// any order of its dimensions
inline int check(const Tensor& t, const char* name, Py_ssize_t k = -1, bool dense = false) {
  if (!t.device().is_cuda())
    throw py::type_error(at_index(name, k) + " must be a GPU tensor, got device " + t.device().str());
  const int code = dtype_code(t);
  if (code < 0)
    throw py::type_error(at_index(name, k) + " must be float32, float16 or bfloat16, got " +
                         c10::toString(t.scalar_type()));
  if (t.layout() != at::kStrided || !(t.is_contiguous() || (dense && t.is_non_overlapping_and_dense())))
    throw py::value_error(at_index(name, k) +
                          (dense ? " must be contiguous or a permutation of a contiguous tensor"
                                 : " must be contiguous"));
  return code;
}

// that the elements of two such tensors of one size lie in the same order
inline void check_order(const Tensor& t, const Tensor& by, const char* name, Py_ssize_t k) {
  if (t.is_contiguous() && by.is_contiguous()) return;
  bool same = t.sizes() == by.sizes();
  for (int64_t d = 0; same && d < t.dim(); ++d)
    same = t.size(d) <= 1 || t.stride(d) == by.stride(d);
  if (!same) throw py::value_error(at_index(name, k) + " must have the strides of its item's others");
}

inline void check_device(const Tensor& t, const c10::Device& dev, const char* name, Py_ssize_t k = -1) {
  if (t.device() != dev)
    throw py::type_error(at_index(name, k) + " must be a tensor on " + dev.str() + ", got " +
                         t.device().str());
}

inline void check_sign(const Tensor& t, const char* name, Py_ssize_t k = -1) {
  // (its memory holds the values with the other sign)
  TORCH_CHECK_NOT_IMPLEMENTED(!t.is_neg(), at_index(name, k), " is a view with its sign turned: use resolve_neg()");
}

// A gradient may arrive as a view with its sign turned, as from a complex number's conjugate.
inline Tensor settled(const Tensor& t) { return t.is_neg() ? t.resolve_neg() : t; }

// any_sign: a view with its sign turned will do
inline const Tensor& unpack(PyObject* o, const char* name, Py_ssize_t k = -1, bool any_sign = false) {
  if (!THPVariable_Check(o)) throw py::type_error(at_index(name, k) + " must be a torch.Tensor");
  const Tensor& t = THPVariable_Unpack(o);
  // (it would be left out of the results: these calls do not pass torch's dispatcher)
  TORCH_CHECK_NOT_IMPLEMENTED(!t._fw_grad(/*level=*/0).defined(), at_index(name, k),
                              " has a forward-mode tangent: forward-mode derivatives of the "
                              "training operators are not available");
  if (!any_sign) check_sign(t, name, k);
  return t;
}

// A trace would hold this call's results as constants and follow no new inputs.
inline void check_tracing(const char* what) {
  using c10::impl::TorchDispatchModeTLS;
  const bool tracing =
      torch::jit::tracer::isTracing() ||
      (c10::impl::dispatch_mode_enabled() &&
       TorchDispatchModeTLS::get_mode(c10::impl::TorchDispatchModeKey::PROXY).has_value());
  TORCH_CHECK_NOT_IMPLEMENTED(!tracing, what, " cannot be recorded by a tracer (torch.jit.trace, "
                              "make_fx)");
}

// a list or tuple of tensors
struct List {
  py::object fast;
  const char* name;
  bool any_sign;
  Py_ssize_t size = 0;
  List(const py::object& o, const char* name_, bool any_sign_ = false) : name(name_), any_sign(any_sign_) {
    if (THPVariable_Check(o.ptr()) || !(PyList_Check(o.ptr()) || PyTuple_Check(o.ptr())))
      throw py::type_error(std::string(name) + " must be a list or tuple of tensors");
    fast = o;
    size = PySequence_Fast_GET_SIZE(o.ptr());
  }
  const Tensor& operator[](Py_ssize_t k) const {
    return unpack(PySequence_Fast_GET_ITEM(fast.ptr(), k), name, k, any_sign);
  }
  bool none(Py_ssize_t k) const { return PySequence_Fast_GET_ITEM(fast.ptr(), k) == Py_None; }
};

inline void* stream_of(const c10::Device& dev) {
  return c10::hip::getCurrentHIPStream(dev.index()).stream();
}

inline void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Outputs and scratch on the current device, straight from torch's allocator: a
// call is as long as its host work where the tensors are small, and at::empty
// takes 0.3 us more of it each.
inline Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const c10::Device& dev) {
  return at::detail::empty_cuda(sizes, type, dev, std::nullopt);
}
inline c10::DataPtr scratch(size_t bytes) { return c10::GetAllocator(c10::kCUDA)->allocate(bytes); }

// A backward pass under capture ends in its inputs' nodes.  Where one of them was
// made on the default stream, by an eager graph that still lives, that stream
// would be made to wait for the capturing one, which HIP does not allow and the
// process does not survive.  So the forward of such a pass is refused.  (Streams
// are compared by number: torch gives them a device type of its own.)
inline void check_capture(const torch::autograd::edge_list& edges, const c10::Device& dev, const char* what) {
  if (c10::hip::currentStreamCaptureStatusMayInitCtx() == c10::hip::CaptureStatus::None) return;
  const c10::StreamId eager = c10::hip::getDefaultHIPStream(dev.index()).id();
  for (const auto& edge : edges) {
    if (!edge.function) continue;
    const auto stream = edge.function->stream();
    TORCH_CHECK(!stream || stream->id() != eager, what, ": captured with gradients, but the node ",
                edge.function->name(), " of an input belongs to the default stream: let go of "
                "graphs that were made of it outside the capture, or use torch.no_grad()");
  }
}

inline Tensor optional(const py::object& o, const char* name) {
  if (o.is_none()) return Tensor();
  return unpack(o.ptr(), name);
}

// the entry points of bind_block.cpp
void add_block(py::module_& m);

}  // namespace ssim_bind
