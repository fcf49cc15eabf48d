// bind.cpp -- the training operators on torch tensors: checks, outputs and
// scratch from torch's caching allocator, and the calls of the C ABI
// (ssim_train_amd.h) on torch's current stream of the tensors' device.
//
// A module of its own in C++ and not ctypes calls: a step over 160 tensors
// looks at some 800 of them, and a small network's joint takes the GPU less
// time than a Python autograd function takes to be recorded.

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
using at::Tensor;

namespace {

std::string text(int code) {
  return std::string(ssim_train_strerror(code)) + " (code " + std::to_string(code) + ")";
}

// Python callers get the package's TrainError
void raise(int code, const char* where) {
  py::object type = py::module_::import("ssim_loss_amd.train").attr("TrainError");
  py::object error = type(code, where);
  PyErr_SetObject(type.ptr(), error.ptr());
  throw py::error_already_set();
}

std::string at_index(const char* name, Py_ssize_t k) {
  return k < 0 ? std::string(name) : std::string(name) + "[" + std::to_string(k) + "]";
}

int dtype_code(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return SSIM_DTYPE_F32;
    case at::kHalf: return SSIM_DTYPE_F16;
    case at::kBFloat16: return SSIM_DTYPE_BF16;
    default: return -1;
  }
}

// a GPU tensor of one of the three types, contiguous or (dense) without gaps in
// any order of its dimensions
int check(const Tensor& t, const char* name, Py_ssize_t k = -1, bool dense = false) {
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
void check_order(const Tensor& t, const Tensor& by, const char* name, Py_ssize_t k) {
  if (t.is_contiguous() && by.is_contiguous()) return;
  bool same = t.sizes() == by.sizes();
  for (int64_t d = 0; same && d < t.dim(); ++d)
    same = t.size(d) <= 1 || t.stride(d) == by.stride(d);
  if (!same) throw py::value_error(at_index(name, k) + " must have the strides of its item's others");
}

void check_device(const Tensor& t, const c10::Device& dev, const char* name, Py_ssize_t k = -1) {
  if (t.device() != dev)
    throw py::type_error(at_index(name, k) + " must be a tensor on " + dev.str() + ", got " +
                         t.device().str());
}

const Tensor& unpack(PyObject* o, const char* name, Py_ssize_t k = -1) {
  if (!THPVariable_Check(o)) throw py::type_error(at_index(name, k) + " must be a torch.Tensor");
  const Tensor& t = THPVariable_Unpack(o);
  // (it would be left out of the results: these calls do not pass torch's dispatcher)
  TORCH_CHECK_NOT_IMPLEMENTED(!t._fw_grad(/*level=*/0).defined(), at_index(name, k),
                              " has a forward-mode tangent: forward-mode derivatives of the "
                              "training operators are not available");
  return t;
}

// A trace would hold this call's results as constants and follow no new inputs.
void check_tracing(const char* what) {
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
  Py_ssize_t size = 0;
  List(const py::object& o, const char* name_) : name(name_) {
    if (THPVariable_Check(o.ptr()) || !(PyList_Check(o.ptr()) || PyTuple_Check(o.ptr())))
      throw py::type_error(std::string(name) + " must be a list or tuple of tensors");
    fast = o;
    size = PySequence_Fast_GET_SIZE(o.ptr());
  }
  const Tensor& operator[](Py_ssize_t k) const {
    return unpack(PySequence_Fast_GET_ITEM(fast.ptr(), k), name, k);
  }
  bool none(Py_ssize_t k) const { return PySequence_Fast_GET_ITEM(fast.ptr(), k) == Py_None; }
};

void* stream_of(const c10::Device& dev) {
  return c10::hip::getCurrentHIPStream(dev.index()).stream();
}

void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Outputs and scratch on the current device, straight from torch's allocator: a
// call is as long as its host work where the tensors are small, and at::empty
// takes 0.3 us more of it each.
Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const c10::Device& dev) {
  return at::detail::empty_cuda(sizes, type, dev, std::nullopt);
}
c10::DataPtr scratch(size_t bytes) { return c10::GetAllocator(c10::kCUDA)->allocate(bytes); }

// ---- clipping
Tensor clip(const py::object& grads_, double max_norm, const py::object& out_, bool scales) {
  check_tracing(scales ? "clip_grads_" : "grad_norm");
  const List grads(grads_, "grads");
  const bool in_place = out_.is_none();
  const List out(in_place ? grads_ : out_, "out");
  if (out.size != grads.size) throw py::value_error("out must have as many tensors as grads");
  if (grads.size == 0) throw py::value_error("grads must hold at least one tensor");
  if (scales && !(max_norm >= 0.0 && max_norm <= 1.7976931348623157e308))
    throw py::value_error("max_norm must be a number >= 0");
  std::vector<ssim_clip_item> items(grads.size);
  const c10::Device dev = grads[0].device();
  for (Py_ssize_t k = 0; k < grads.size; ++k) {
    const Tensor& g = grads[k];
    ssim_clip_item& it = items[k];
    it.dtype = check(g, "grads", k, true);
    check_device(g, dev, "grads", k);
    it.grad = g.const_data_ptr();
    it.n = g.numel();
    it.reserved = 0;
    it.out = nullptr;
    if (!scales) continue;
    const Tensor& o = out[k];
    if (!in_place) {
      check_device(o, dev, "out", k);
      if (check(o, "out", k, true) != it.dtype)
        throw py::type_error(at_index("out", k) + " must have its gradient's dtype");
      if (o.sizes() != g.sizes())
        throw py::value_error(at_index("out", k) + " must have its gradient's shape");
      check_order(o, g, "out", k);
    }
    it.out = o.data_ptr();
  }
  const c10::DeviceGuard guard(dev);
  Tensor norm = fresh({}, at::kFloat, dev);
  const c10::DataPtr ws = scratch(ssim_update_workspace_bytes());
  float* n = norm.data_ptr<float>();
  const int rc = scales ? ssim_clip_grads(items.data(), grads.size, max_norm, n, ws.get(),
                                          stream_of(dev))
                        : ssim_grad_norm(items.data(), grads.size, n, ws.get(), stream_of(dev));
  if (rc != SSIM_OK) raise(rc, scales ? "ssim_clip_grads" : "ssim_grad_norm");
  if (scales)
    for (Py_ssize_t k = 0; k < out.size; ++k) written(out[k]);
  return norm;
}

Tensor clip_grads(const py::object& grads, double max_norm, const py::object& out) {
  return clip(grads, max_norm, out, true);
}
Tensor grad_norm(const py::object& grads) { return clip(grads, 0.0, py::none(), false); }

// ---- AdamW
py::object adamw_step(const py::object& grads_, const py::object& params_, const py::object& m_,
                      const py::object& v_, const py::object& masters_, const py::object& step_,
                      const py::object& lr, double beta1, double beta2, double eps,
                      double weight_decay, const py::object& max_norm) {
  check_tracing("AdamW.step");
  const List grads(grads_, "grads"), params(params_, "params"), m(m_, "exp_avgs"),
      v(v_, "exp_avg_sqs");
  const bool has_masters = !masters_.is_none();
  const List masters(has_masters ? masters_ : params_, "masters");
  if (grads.size != params.size)
    throw py::value_error("grads must have as many entries as params");
  if (m.size != params.size || v.size != params.size || masters.size != params.size)
    throw py::value_error("exp_avgs, exp_avg_sqs and masters must have as many tensors as params");
  if (params.size == 0) throw py::value_error("params must hold at least one tensor");
  const c10::Device dev = params[0].device();
  std::vector<ssim_adamw_item> items;
  items.reserve(params.size);
  for (Py_ssize_t k = 0; k < params.size; ++k) {
    if (grads.none(k)) continue;
    const Tensor &g = grads[k], &p = params[k], &mk = m[k], &vk = v[k];
    ssim_adamw_item it;
    it.grad_dtype = check(g, "grads", k, true);
    it.param_dtype = check(p, "params", k, true);
    const int cm = check(mk, "exp_avgs", k, true), cv = check(vk, "exp_avg_sqs", k, true);
    if (it.grad_dtype != it.param_dtype && it.grad_dtype != SSIM_DTYPE_F32)
      throw py::type_error(at_index("grads", k) + " must be float32 or have its parameter's dtype");
    if (cm != SSIM_DTYPE_F32 || cv != SSIM_DTYPE_F32)
      throw py::type_error(at_index("exp_avgs and exp_avg_sqs", k) + " must be float32");
    it.n = p.numel();
    if (g.sizes() != p.sizes() || mk.numel() != it.n || vk.numel() != it.n)
      throw py::value_error(at_index("grads, exp_avgs and exp_avg_sqs", k) +
                            " must have their parameter's shape");
    check_order(g, p, "grads", k);
    check_order(mk, p, "exp_avgs", k);
    check_order(vk, p, "exp_avg_sqs", k);
    check_device(g, dev, "grads", k);
    check_device(p, dev, "params", k);
    check_device(mk, dev, "exp_avgs", k);
    check_device(vk, dev, "exp_avg_sqs", k);
    it.grad = g.const_data_ptr();
    it.param = p.data_ptr();
    it.exp_avg = (float*)mk.data_ptr();
    it.exp_avg_sq = (float*)vk.data_ptr();
    it.master = nullptr;
    if (has_masters && !masters.none(k)) {
      const Tensor& w = masters[k];
      if (check(w, "masters", k, true) != SSIM_DTYPE_F32)
        throw py::type_error(at_index("masters", k) + " must be float32");
      if (w.numel() != it.n)
        throw py::value_error(at_index("masters", k) + " must have its parameter's shape");
      check_order(w, p, "masters", k);
      check_device(w, dev, "masters", k);
      it.master = (float*)w.data_ptr();
    }
    items.push_back(it);
  }
  const Tensor& step = unpack(step_.ptr(), "step");
  if (step.scalar_type() != at::kLong || step.numel() != 2 || !step.is_contiguous())
    throw py::type_error("step must be two int64");
  check_device(step, dev, "step");
  ssim_adamw_options o;
  o.lr = 0.0;
  o.lr_device = nullptr;
  if (THPVariable_Check(lr.ptr())) {
    const Tensor& t = unpack(lr.ptr(), "lr");
    if (check(t, "lr") != SSIM_DTYPE_F32 || t.numel() != 1)
      throw py::type_error("lr must be a number or one float32 on the parameters' device");
    check_device(t, dev, "lr");
    o.lr_device = t.const_data_ptr<float>();
  } else {
    o.lr = lr.cast<double>();
  }
  o.beta1 = beta1;
  o.beta2 = beta2;
  o.eps = eps;
  o.weight_decay = weight_decay;
  const bool clips = !max_norm.is_none();
  o.max_norm = clips ? max_norm.cast<double>() : HUGE_VAL;
  const c10::DeviceGuard guard(dev);
  Tensor norm;
  if (clips) norm = fresh({}, at::kFloat, dev);
  const c10::DataPtr ws = scratch(ssim_update_workspace_bytes());
  const int rc =
      ssim_adamw_step(items.data(), (int64_t)items.size(), &o, step.data_ptr<int64_t>(),
                      clips ? norm.data_ptr<float>() : nullptr, ws.get(), stream_of(dev));
  if (rc != SSIM_OK) raise(rc, "ssim_adamw_step");
  for (Py_ssize_t k = 0; k < params.size; ++k) {
    if (grads.none(k)) continue;
    written(params[k]);
    written(m[k]);
    written(v[k]);
    if (has_masters && !masters.none(k)) written(masters[k]);
  }
  written(step);
  if (!clips) return py::none();
  return py::cast(norm);
}

// ---- the joint between two blocks
ssim_block_norm_inputs inputs_of(const Tensor& x, const Tensor& branch, const Tensor& gate,
                                 const Tensor& scale, const Tensor& post, const Tensor& pre,
                                 double eps, int act) {
  ssim_block_norm_inputs in;
  auto weight = [](const Tensor& t) { return t.defined() ? t.const_data_ptr<float>() : nullptr; };
  in.x = x.const_data_ptr();
  in.branch = branch.const_data_ptr();
  in.gate = gate.defined() ? gate.const_data_ptr() : nullptr;
  in.scale = weight(scale);
  in.post_weight = weight(post);
  in.pre_weight = weight(pre);
  in.width = x.size(-1);
  in.rows = x.numel() / in.width;
  const int64_t gates = gate.defined() ? gate.numel() / in.width : 0;
  in.gate_rows = gates > 0 && in.rows > 0 ? in.rows / gates : 1;
  in.eps = eps;
  in.x_dtype = dtype_code(x);
  in.branch_dtype = dtype_code(branch);
  in.gate_act = act;
  in.reserved = 0;
  return in;
}

void forward_into(const ssim_block_norm_inputs& in, const Tensor& residual, const Tensor& normed,
                  float* stats, const c10::Device& dev) {
  const int rc = ssim_block_norm_forward(&in, residual.data_ptr(), normed.data_ptr(), stats,
                                         stream_of(dev));
  if (rc != SSIM_OK) raise(rc, "ssim_block_norm_forward");
}

// A backward pass under capture ends in its inputs' nodes.  Where one of them was
// made on the default stream, by an eager graph that still lives, that stream
// would be made to wait for the capturing one, which HIP does not allow and the
// process does not survive.  So the forward of such a pass is refused.  (Streams
// are compared by number: torch gives them a device type of its own.)
void check_capture(const torch::autograd::edge_list& edges, const c10::Device& dev) {
  if (c10::hip::currentStreamCaptureStatusMayInitCtx() == c10::hip::CaptureStatus::None) return;
  const c10::StreamId eager = c10::hip::getDefaultHIPStream(dev.index()).id();
  for (const auto& edge : edges) {
    if (!edge.function) continue;
    const auto stream = edge.function->stream();
    TORCH_CHECK(!stream || stream->id() != eager, "block_norm: captured with gradients, but the node ",
                edge.function->name(), " of an input belongs to the default stream: let go of "
                "graphs that were made of it outside the capture, or use torch.no_grad()");
  }
}

// The joint's node in an autograd graph.  A node itself, not a Function with a
// context: that recorded a call in 2.8 us more than this.
struct BlockNormBackward : torch::autograd::Node {
  static constexpr int kTensors = 7;  // x, branch, gate, scale, post and pre weight; the row's roots
  torch::autograd::SavedVariable saved[kTensors];
  double eps = 0;
  int act = 0;

  std::string name() const override { return "BlockNormBackward"; }

  void release_variables() override {
    std::lock_guard<std::mutex> lock(mutex_);
    for (auto& s : saved) s.reset_data();
  }

  torch::autograd::variable_list apply(torch::autograd::variable_list&& upstream) override {
    std::lock_guard<std::mutex> lock(mutex_);
    TORCH_CHECK(!at::GradMode::is_enabled(),
                "block_norm: the gradient of the gradient is not available (create_graph=True)");
    Tensor in_[kTensors];
    for (int k = 0; k < kTensors; ++k) in_[k] = saved[k].unpack();
    const Tensor &x = in_[0], &stats = in_[6];
    const c10::Device dev = x.device();
    const c10::DeviceGuard guard(dev);
    const ssim_block_norm_inputs in =
        inputs_of(x, in_[1], in_[2], in_[3], in_[4], in_[5], eps, act);
    torch::autograd::variable_list out(kTensors - 1);
    Tensor dr = upstream[0], dh = upstream[1];
    if (!dr.defined() && !dh.defined()) return out;
    auto wanted = [&](int k) -> void* {
      if (!in_[k].defined() || !task_should_compute_output(k)) return nullptr;
      out[k] = in.rows > 0 ? fresh(in_[k].sizes(), in_[k].scalar_type(), dev)
                           : at::zeros(in_[k].sizes(), in_[k].options());
      return out[k].data_ptr();
    };
    ssim_block_norm_grads grads;
    grads.x = wanted(0);
    grads.branch = wanted(1);
    grads.gate = wanted(2);
    grads.scale = (float*)wanted(3);
    grads.post_weight = (float*)wanted(4);
    grads.pre_weight = (float*)wanted(5);
    if (in.rows == 0) return out;
    if (dr.defined()) dr = dr.contiguous();
    if (dh.defined()) dh = dh.contiguous();
    const c10::DataPtr ws = scratch(ssim_block_norm_workspace_bytes(&in));
    const int rc = ssim_block_norm_backward(
        &in, stats.const_data_ptr<float>(), dr.defined() ? dr.const_data_ptr() : nullptr,
        dh.defined() ? dh.const_data_ptr() : nullptr, &grads, ws.get(), stream_of(dev));
    TORCH_CHECK(rc == SSIM_OK, "ssim_block_norm_backward: ", text(rc));
    return out;
  }
};

Tensor optional(const py::object& o, const char* name) {
  if (o.is_none()) return Tensor();
  return unpack(o.ptr(), name);
}

py::tuple block_norm(const py::object& x_, const py::object& branch_, const py::object& gate_,
                     const py::object& scale_, const py::object& post_, const py::object& pre_,
                     double eps, int act) {
  check_tracing("block_norm");
  const Tensor x = unpack(x_.ptr(), "x"), branch = unpack(branch_.ptr(), "branch"),
               gate = optional(gate_, "gate"), scale = optional(scale_, "scale"),
               post = optional(post_, "post_weight"), pre = optional(pre_, "pre_weight");
  const int cx = check(x, "x"), cb = check(branch, "branch");
  const c10::Device dev = x.device();
  check_device(branch, dev, "branch");
  if (x.dim() < 1) throw py::value_error("x must have at least one dimension");
  if (x.sizes() != branch.sizes()) throw py::value_error("x and branch must have the same shape");
  if (cx != cb && cx != SSIM_DTYPE_F32)
    throw py::type_error("x must be float32 or have branch's dtype");
  const int64_t width = x.size(-1);
  if (width < 1 || width > SSIM_BLOCK_NORM_MAX_WIDTH)
    throw py::value_error("the last dimension must have 1 to " +
                          std::to_string(SSIM_BLOCK_NORM_MAX_WIDTH) + " elements, got " +
                          std::to_string(width));
  if (!(eps >= 0.0 && eps <= 1.7976931348623157e308))
    throw py::value_error("eps must be a number >= 0");
  bool wants = x.requires_grad() || branch.requires_grad();
  if (gate.defined()) {
    if (check(gate, "gate") != cb) throw py::type_error("gate must have branch's dtype");
    check_device(gate, dev, "gate");
    // x's shape, or ones in the place of its last few leading dimensions
    bool ok = gate.dim() == x.dim() && gate.size(-1) == width, ones = false;
    for (int64_t k = 0; ok && k + 1 < x.dim(); ++k) {
      if (gate.size(k) == x.size(k) && !(ones && x.size(k) != 1)) continue;
      ok = gate.size(k) == 1;
      ones = true;
    }
    if (!ok)
      throw py::value_error(
          "gate must have x's shape, or x's shape with ones in the place of the last few "
          "dimensions before the width");
    wants |= gate.requires_grad();
  }
  const struct {
    const Tensor& t;
    const char* name;
  } weights[] = {{scale, "scale"}, {post, "post_weight"}, {pre, "pre_weight"}};
  for (const auto& w : weights) {
    if (!w.t.defined()) continue;
    if (check(w.t, w.name) != SSIM_DTYPE_F32)
      throw py::type_error(std::string(w.name) + " must be float32");
    check_device(w.t, dev, w.name);
    if (w.t.dim() != 1 || w.t.size(0) != width)
      throw py::value_error(std::string(w.name) + " must have one value for each of the width");
    wants |= w.t.requires_grad();
  }
  const c10::DeviceGuard guard(dev);
  const Tensor* tensors[] = {&x, &branch, &gate, &scale, &post, &pre};
  torch::autograd::edge_list edges(BlockNormBackward::kTensors - 1);
  wants = wants && at::GradMode::is_enabled();
  if (wants) {
    for (size_t k = 0; k < edges.size(); ++k)
      if (tensors[k]->defined() && tensors[k]->requires_grad())
        edges[k] = torch::autograd::impl::gradient_edge(*tensors[k]);
    check_capture(edges, dev);
  }
  const ssim_block_norm_inputs in = inputs_of(x, branch, gate, scale, post, pre, eps, act);
  Tensor residual = fresh(x.sizes(), x.scalar_type(), dev);
  Tensor normed = fresh(branch.sizes(), branch.scalar_type(), dev);
  Tensor stats;
  if (wants) stats = fresh({in.rows, 2}, at::kFloat, dev);
  forward_into(in, residual, normed, wants ? stats.data_ptr<float>() : nullptr, dev);
  if (wants) {
    std::shared_ptr<BlockNormBackward> node(new BlockNormBackward(), torch::autograd::deleteNode);
    for (size_t k = 0; k < edges.size(); ++k)
      if (tensors[k]->defined()) node->saved[k] = torch::autograd::SavedVariable(*tensors[k], false);
    node->saved[6] = torch::autograd::SavedVariable(stats, false);
    node->eps = eps;
    node->act = act;
    node->set_next_edges(std::move(edges));
    torch::autograd::set_history(residual, node);
    torch::autograd::set_history(normed, node);
  }
  return py::make_tuple(residual, normed);
}

}  // namespace

PYBIND11_MODULE(_bind, m) {
  if (ssim_train_abi_version() != SSIM_TRAIN_ABI_VERSION)
    throw py::import_error("the training library implements ABI version " +
                           std::to_string(ssim_train_abi_version()) + ", its binding version " +
                           std::to_string(SSIM_TRAIN_ABI_VERSION) + ": rebuild it");
  m.def("clip_grads", &clip_grads);
  m.def("grad_norm", &grad_norm);
  m.def("adamw_step", &adamw_step);
  m.def("block_norm", &block_norm);
  m.def("abi_version", &ssim_train_abi_version);
  m.def("strerror", &ssim_train_strerror);
}
