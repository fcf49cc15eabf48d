// bind_block.cpp -- what lies inside a block of an image network, on torch
// tensors: rotary positions, attention and the gated layer, each a node of its
// own in an autograd graph.

#include "bind_common.hpp"

namespace ssim_bind {

namespace {

using torch::autograd::SavedVariable;
using torch::autograd::variable_list;

constexpr const char* kNoSecond = ": the gradient of the gradient is not available (create_graph=True)";

// Tensors as the nodes of their gradients' graph.
torch::autograd::edge_list edges_of(std::initializer_list<const Tensor*> tensors) {
  torch::autograd::edge_list edges;
  for (const Tensor* t : tensors)
    edges.push_back(t->defined() && t->requires_grad() ? torch::autograd::impl::gradient_edge(*t)
                                                       : torch::autograd::Edge());
  return edges;
}
bool wants_gradient(std::initializer_list<const Tensor*> tensors) {
  if (!at::GradMode::is_enabled()) return false;
  for (const Tensor* t : tensors)
    if (t->defined() && t->requires_grad()) return true;
  return false;
}

// GPU tensors of one of the three types, any strides
int check_strided(const Tensor& t, const char* name) {
  if (!t.device().is_cuda()) throw py::type_error(std::string(name) + " must be a GPU tensor, got device " + t.device().str());
  const int code = dtype_code(t);
  if (code < 0)
    throw py::type_error(std::string(name) + " must be float32, float16 or bfloat16, got " + c10::toString(t.scalar_type()));
  if (t.layout() != at::kStrided) throw py::value_error(std::string(name) + " must be a strided tensor");
  if (t.dim() != 4) throw py::value_error(std::string(name) + " must have 4 dimensions: batch, tokens, heads, dim");
  return code;
}

// (an expanded tensor has more heads than memory, and than the ABI's ints count)
constexpr int64_t kMostHeads = 65536;
[[noreturn]] void refuse_heads() { throw py::value_error("there must be at most " + std::to_string(kMostHeads) + " heads"); }

Tensor dense_copy(const Tensor& t, const c10::Device& dev) {
  const at::NoGradGuard no_grad;
  Tensor c = fresh(t.sizes(), t.scalar_type(), dev);
  c.copy_(t);
  return c;
}
// the first `n` strides, 0 where a dimension has one entry
void strides_of(const Tensor& t, int64_t* to, int n) {
  for (int k = 0; k < n; ++k) to[k] = t.size(k) > 1 ? t.stride(k) : 0;
}

// ---------------------------------------------------------------- rotary positions
struct RotaryPlan {
  std::vector<int> axes;
  double base = 0;
  int pairs = 0;
};

Tensor rows_in_place(const Tensor& t, const c10::Device& dev) {
  return t.size(3) <= 1 || t.stride(3) == 1 ? t : dense_copy(t, dev);
}

// (q, k) turned; k may be undefined
std::pair<Tensor, Tensor> turn(const Tensor& q_, const Tensor& k_, const Tensor& positions, const RotaryPlan& plan,
                               bool inverse, const c10::Device& dev, int& rc) {
  const Tensor q = rows_in_place(q_, dev), k = k_.defined() ? rows_in_place(k_, dev) : Tensor();
  ssim_rotary_inputs in = {};
  in.q = q.const_data_ptr();
  in.positions = positions.const_data_ptr();
  strides_of(q, in.q_stride, 3);
  in.batch = q.size(0);
  in.tokens = q.size(1);
  in.q_heads = (int)q.size(2);
  in.dim = (int)q.size(3);
  if (k.defined()) {
    in.k = k.const_data_ptr();
    strides_of(k, in.k_stride, 3);
    in.k_heads = (int)k.size(2);
  }
  const int64_t lead = positions.dim() - 2;  // 0: the same for all of the batch
  in.position_stride[0] = lead && positions.size(0) > 1 ? positions.stride(0) : 0;
  in.position_stride[1] = positions.size(lead) > 1 ? positions.stride(lead) : 0;
  in.axes = (int)plan.axes.size();
  for (int a = 0; a < in.axes; ++a) in.axis_size[a] = plan.axes[a];
  in.pairs = plan.pairs;
  in.position_type = positions.scalar_type() == at::kFloat ? SSIM_POSITION_F32
                     : positions.scalar_type() == at::kInt ? SSIM_POSITION_I32
                                                           : SSIM_POSITION_I64;
  in.dtype = dtype_code(q);
  in.inverse = inverse;
  in.base = plan.base;
  Tensor q_out = fresh(q.sizes(), q.scalar_type(), dev), k_out;
  if (k.defined()) k_out = fresh(k.sizes(), k.scalar_type(), dev);
  rc = SSIM_OK;
  // (a tensor without elements has no memory to name)
  if (q.numel() > 0) rc = ssim_rotary(&in, q_out.data_ptr(), k.defined() ? k_out.data_ptr() : nullptr, stream_of(dev));
  return {q_out, k_out};
}

struct RotaryBackward : torch::autograd::Node {
  SavedVariable positions;
  RotaryPlan plan;

  std::string name() const override { return "RotaryBackward"; }

  void release_variables() override {
    std::lock_guard<std::mutex> lock(mutex_);
    positions.reset_data();
  }

  variable_list apply(variable_list&& upstream) override {
    std::lock_guard<std::mutex> lock(mutex_);
    TORCH_CHECK(!at::GradMode::is_enabled(), "rotary", kNoSecond);
    const Tensor at_ = positions.unpack();
    const c10::Device dev = at_.device();
    const c10::DeviceGuard guard(dev);
    variable_list out(num_outputs());
    std::vector<int> which;
    for (int k = 0; k < (int)num_outputs(); ++k)
      if (upstream[k].defined() && task_should_compute_output(k)) which.push_back(k);
    if (which.empty()) return out;
    int rc = SSIM_OK;
    auto turned = turn(settled(upstream[which[0]]), which.size() > 1 ? settled(upstream[which[1]]) : Tensor(), at_,
                       plan, true, dev, rc);
    TORCH_CHECK(rc == SSIM_OK, "ssim_rotary: ", text(rc));
    out[which[0]] = turned.first;
    if (which.size() > 1) out[which[1]] = turned.second;
    return out;
  }
};

py::tuple rotary(const py::object& q_, const py::object& k_, const py::object& positions_, const py::object& axes_,
                 double base, int pairs) {
  check_tracing("rotary");
  const Tensor q = unpack(q_.ptr(), "q"), k = optional(k_, "k");
  Tensor positions = unpack(positions_.ptr(), "positions");
  const int code = check_strided(q, "q");
  const c10::Device dev = q.device();
  if (k.defined()) {
    if (check_strided(k, "k") != code) throw py::type_error("k must have q's dtype");
    check_device(k, dev, "k");
    if (k.size(0) != q.size(0) || k.size(1) != q.size(1) || k.size(3) != q.size(3))
      throw py::value_error("k must have q's batch, tokens and dim");
  }
  if (q.size(2) < 1 || q.size(3) < 1 || (k.defined() && k.size(2) < 1))
    throw py::value_error("q and k must have at least one head of one element");
  if (q.size(2) > kMostHeads || (k.defined() && k.size(2) > kMostHeads)) refuse_heads();
  RotaryPlan plan;
  plan.base = base;
  plan.pairs = pairs;
  if (!(base > 0.0 && base <= 1.7976931348623157e308)) throw py::value_error("base must be a number > 0");
  const int64_t dim = q.size(3);
  int64_t sum = 0;
  for (const auto& a : axes_) {
    const int64_t size = py::cast<int64_t>(a);
    if (size < 2 || size % 2 != 0 || size > dim) throw py::value_error("axes must be even sizes of 2 to dim elements");
    sum += size;
    plan.axes.push_back((int)size);
  }
  if (plan.axes.empty() || plan.axes.size() > SSIM_ROTARY_MAX_AXES || sum > dim)
    throw py::value_error("axes must be 1 to " + std::to_string(SSIM_ROTARY_MAX_AXES) + " sizes that add up to at most dim");
  if (dim > SSIM_ROTARY_MAX_DIM)
    throw py::value_error("dim must be at most " + std::to_string(SSIM_ROTARY_MAX_DIM));
  check_device(positions, dev, "positions");
  const auto type = positions.scalar_type();
  if (type != at::kFloat && type != at::kInt && type != at::kLong)
    throw py::type_error("positions must be float32, int32 or int64");
  TORCH_CHECK_NOT_IMPLEMENTED(!(positions.requires_grad() && at::GradMode::is_enabled()),
                              "rotary: the gradient of positions is not available");
  const int64_t lead = positions.dim() - 2;
  if (positions.layout() != at::kStrided || (lead != 0 && lead != 1) ||
      (lead == 1 && positions.size(0) != q.size(0) && positions.size(0) != 1) || positions.size(lead) != q.size(1) ||
      positions.size(lead + 1) != (int64_t)plan.axes.size())
    throw py::value_error("positions must be [tokens, axes] or [batch, tokens, axes]");
  const c10::DeviceGuard guard(dev);
  if (positions.size(lead + 1) > 1 && positions.stride(lead + 1) != 1) positions = dense_copy(positions, dev);
  const bool wants = wants_gradient({&q, &k});
  torch::autograd::edge_list edges;
  if (wants) {
    edges = k.defined() ? edges_of({&q, &k}) : edges_of({&q});
    check_capture(edges, dev, "rotary");
  }
  int rc = SSIM_OK;
  auto turned = turn(q, k, positions, plan, false, dev, rc);
  if (rc != SSIM_OK) raise(rc, "ssim_rotary");
  if (wants) {
    std::shared_ptr<RotaryBackward> node(new RotaryBackward(), torch::autograd::deleteNode);
    node->positions = SavedVariable(positions, false);
    node->plan = plan;
    node->set_next_edges(std::move(edges));
    torch::autograd::set_history(turned.first, node);
    if (k.defined()) torch::autograd::set_history(turned.second, node);
  }
  return py::make_tuple(turned.first, k.defined() ? py::cast(turned.second) : py::object(py::none()));
}

// ---------------------------------------------------------------- attention
struct AttentionPlan {
  double scale = 0;
  bool causal = false;
};

// What the kernels can load: rows without gaps at multiples of 16 bytes.
// Tensors that lie otherwise are copied.
Tensor loadable(const Tensor& t, const c10::Device& dev) {
  const int64_t bytes = t.element_size();
  bool ok = t.stride(3) == 1 && (uintptr_t)t.const_data_ptr() % 16 == 0;
  for (int k = 0; ok && k < 3; ++k) ok = t.size(k) <= 1 || t.stride(k) * bytes % 16 == 0;
  if (ok && t.size(1) > 1) ok = t.stride(1) >= t.size(3) && t.stride(1) * bytes < 1 << 24;
  return ok ? t : dense_copy(t, dev);
}

struct AttentionCall {
  ssim_attention_inputs in = {};
  Tensor q, k, v;  // held while the call runs

  AttentionCall(const Tensor& q_, const Tensor& k_, const Tensor& v_, const Tensor& q_lengths, const Tensor& k_lengths,
                const AttentionPlan& plan, const c10::Device& dev)
      : q(loadable(q_, dev)), k(loadable(k_, dev)), v(loadable(v_, dev)) {
    in.q = q.const_data_ptr();
    in.k = k.const_data_ptr();
    in.v = v.const_data_ptr();
    if (q_lengths.defined()) in.q_lengths = q_lengths.const_data_ptr<int32_t>();
    if (k_lengths.defined()) in.k_lengths = k_lengths.const_data_ptr<int32_t>();
    strides_of(q, in.q_stride, 3);
    strides_of(k, in.k_stride, 3);
    strides_of(v, in.v_stride, 3);
    in.batch = q.size(0);
    in.q_tokens = q.size(1);
    in.k_tokens = k.size(1);
    in.heads = (int)q.size(2);
    in.kv_heads = (int)k.size(2);
    in.dim = (int)q.size(3);
    in.causal = plan.causal;
    in.dtype = dtype_code(q);
    in.scale = plan.scale;
  }
};

struct AttentionBackward : torch::autograd::Node {
  static constexpr int kTensors = 8;  // q, k, v, the lengths, out, lse, rest
  SavedVariable saved[kTensors];
  AttentionPlan plan;

  std::string name() const override { return "AttentionBackward"; }

  void release_variables() override {
    std::lock_guard<std::mutex> lock(mutex_);
    for (auto& s : saved) s.reset_data();
  }

  variable_list apply(variable_list&& upstream) override {
    std::lock_guard<std::mutex> lock(mutex_);
    TORCH_CHECK(!at::GradMode::is_enabled(), "attention", kNoSecond);
    variable_list out(3);
    if (!upstream[0].defined()) return out;
    Tensor t[kTensors];
    for (int k = 0; k < kTensors; ++k) t[k] = saved[k].unpack(shared_from_this());
    const c10::Device dev = t[0].device();
    const c10::DeviceGuard guard(dev);
    void* grads[3] = {};
    for (int k = 0; k < 3; ++k) {
      if (!task_should_compute_output(k)) continue;
      out[k] = fresh(t[k].sizes(), t[k].scalar_type(), dev);
      grads[k] = out[k].data_ptr();
    }
    const AttentionCall call(t[0], t[1], t[2], t[3], t[4], plan, dev);
    Tensor d_out = settled(upstream[0]).contiguous();
    if ((uintptr_t)d_out.const_data_ptr() % 16 != 0) d_out = dense_copy(d_out, dev);
    const c10::DataPtr ws = scratch(ssim_attention_backward_workspace_bytes(&call.in));
    const int rc = ssim_attention_backward(&call.in, t[5].const_data_ptr(), t[6].const_data_ptr<float>(),
                                           t[7].defined() ? t[7].const_data_ptr() : nullptr, d_out.const_data_ptr(), grads[0], grads[1], grads[2], ws.get(), stream_of(dev));
    TORCH_CHECK(rc == SSIM_OK, "ssim_attention_backward: ", text(rc));
    return out;
  }
};

Tensor lengths_of(const py::object& o, const char* name, int64_t batch, const c10::Device& dev) {
  const Tensor t = optional(o, name);
  if (!t.defined()) return t;
  check_device(t, dev, name);
  if (t.scalar_type() != at::kInt) throw py::type_error(std::string(name) + " must be int32");
  if (t.layout() != at::kStrided || t.dim() != 1 || t.size(0) != batch || !t.is_contiguous())
    throw py::value_error(std::string(name) + " must be one contiguous number for each of the batch");
  return t;
}

Tensor attention(const py::object& q_, const py::object& k_, const py::object& v_, const py::object& scale_, bool causal,
                 const py::object& q_lengths_, const py::object& k_lengths_) {
  check_tracing("attention");
  const Tensor q = unpack(q_.ptr(), "q"), k = unpack(k_.ptr(), "k"), v = unpack(v_.ptr(), "v");
  const int code = check_strided(q, "q");
  const c10::Device dev = q.device();
  if (check_strided(k, "k") != code || check_strided(v, "v") != code) throw py::type_error("k and v must have q's dtype");
  check_device(k, dev, "k");
  check_device(v, dev, "v");
  if (k.sizes() != v.sizes()) throw py::value_error("k and v must have the same shape");
  if (k.size(0) != q.size(0) || k.size(3) != q.size(3)) throw py::value_error("k and v must have q's batch and dim");
  if (q.size(2) < 1 || k.size(2) < 1 || q.size(2) % k.size(2) != 0)
    throw py::value_error("q's heads must be a multiple of k's");
  if (q.size(2) > kMostHeads) refuse_heads();
  if (q.size(3) < 8 || q.size(3) > SSIM_ATTENTION_MAX_DIM || q.size(3) % 8 != 0)
    throw py::value_error("dim must be a multiple of 8, to " + std::to_string(SSIM_ATTENTION_MAX_DIM));
  AttentionPlan plan;
  plan.causal = causal;
  plan.scale = scale_.is_none() ? 1.0 / std::sqrt((double)q.size(3)) : scale_.cast<double>();
  if (!(plan.scale > 0.0 && plan.scale <= 1.7976931348623157e308)) throw py::value_error("scale must be a number > 0");
  const Tensor q_lengths = lengths_of(q_lengths_, "query_lengths", q.size(0), dev);
  const Tensor k_lengths = lengths_of(k_lengths_, "key_lengths", q.size(0), dev);
  const c10::DeviceGuard guard(dev);
  const bool wants = wants_gradient({&q, &k, &v});
  torch::autograd::edge_list edges;
  if (wants) {
    edges = edges_of({&q, &k, &v});
    check_capture(edges, dev, "attention");
  }
  const AttentionCall call(q, k, v, q_lengths, k_lengths, plan, dev);
  Tensor out = fresh(q.sizes(), q.scalar_type(), dev), lse, rest;
  if (wants) lse = fresh({q.size(0), q.size(2), q.size(1)}, at::kFloat, dev);
  if (wants && q.scalar_type() != at::kFloat) rest = fresh(q.sizes(), q.scalar_type(), dev);
  const size_t bytes = ssim_attention_workspace_bytes(&call.in);
  const c10::DataPtr ws = bytes ? scratch(bytes) : c10::DataPtr();
  const int rc = ssim_attention_forward(&call.in, out.data_ptr(), wants ? lse.data_ptr<float>() : nullptr,
                                        rest.defined() ? rest.data_ptr() : nullptr, ws.get(), stream_of(dev));
  if (rc != SSIM_OK) raise(rc, "ssim_attention_forward");
  if (wants) {
    std::shared_ptr<AttentionBackward> node(new AttentionBackward(), torch::autograd::deleteNode);
    node->plan = plan;
    node->set_next_edges(std::move(edges));
    torch::autograd::set_history(out, node);
    const Tensor* tensors[] = {&q, &k, &v, &q_lengths, &k_lengths};
    for (int n = 0; n < 5; ++n)
      if (tensors[n]->defined()) node->saved[n] = SavedVariable(*tensors[n], false);
    node->saved[5] = SavedVariable(out, true);
    node->saved[6] = SavedVariable(lse, false);
    if (rest.defined()) node->saved[7] = SavedVariable(rest, false);
  }
  return out;
}

// ---------------------------------------------------------------- the gated layer
ssim_gated_linear_inputs gated_inputs(const Tensor& x, const Tensor& w_gate, const Tensor& w_up, const Tensor& b_gate,
                                      const Tensor& b_up, int act) {
  ssim_gated_linear_inputs in = {};
  in.x = x.const_data_ptr();
  in.w_gate = w_gate.const_data_ptr();
  in.w_up = w_up.const_data_ptr();
  in.b_gate = b_gate.defined() ? b_gate.const_data_ptr() : nullptr;
  in.b_up = b_up.defined() ? b_up.const_data_ptr() : nullptr;
  in.width = w_gate.size(1);
  in.hidden = w_gate.size(0);
  in.rows = x.numel() / in.width;
  in.act = act;
  in.dtype = dtype_code(x);
  return in;
}

struct GatedLinearBackward : torch::autograd::Node {
  static constexpr int kTensors = 7;  // x, the weights, the biases, g, u
  SavedVariable saved[kTensors];
  int act = 0;

  std::string name() const override { return "GatedLinearBackward"; }

  void release_variables() override {
    std::lock_guard<std::mutex> lock(mutex_);
    for (auto& s : saved) s.reset_data();
  }

  variable_list apply(variable_list&& upstream) override {
    std::lock_guard<std::mutex> lock(mutex_);
    TORCH_CHECK(!at::GradMode::is_enabled(), "gated_linear", kNoSecond);
    variable_list out(5);
    if (!upstream[0].defined()) return out;
    Tensor t[kTensors];
    for (int k = 0; k < kTensors; ++k) t[k] = saved[k].unpack();
    const c10::Device dev = t[0].device();
    const c10::DeviceGuard guard(dev);
    const ssim_gated_linear_inputs in = gated_inputs(t[0], t[1], t[2], t[3], t[4], act);
    auto wanted = [&](int k) -> void* {
      if (!t[k].defined() || !task_should_compute_output(k)) return nullptr;
      out[k] = fresh(t[k].sizes(), t[k].scalar_type(), dev);
      return out[k].data_ptr();
    };
    ssim_gated_linear_grads grads;
    grads.x = wanted(0);
    grads.w_gate = wanted(1);
    grads.w_up = wanted(2);
    grads.b_gate = wanted(3);
    grads.b_up = wanted(4);
    const Tensor d_out = settled(upstream[0]).contiguous();
    const c10::DataPtr ws = scratch(ssim_gated_linear_backward_workspace_bytes(&in));
    const int rc = ssim_gated_linear_backward(&in, t[5].const_data_ptr<float>(), t[6].const_data_ptr<float>(),
                                              d_out.const_data_ptr(), &grads, ws.get(), stream_of(dev));
    TORCH_CHECK(rc == SSIM_OK, "ssim_gated_linear_backward: ", text(rc));
    return out;
  }
};

Tensor gated_linear(const py::object& x_, const py::object& w_gate_, const py::object& w_up_, const py::object& b_gate_,
                    const py::object& b_up_, int act) {
  check_tracing("gated_linear");
  const Tensor x = unpack(x_.ptr(), "x"), w_gate = unpack(w_gate_.ptr(), "w_gate"), w_up = unpack(w_up_.ptr(), "w_up"),
               b_gate = optional(b_gate_, "b_gate"), b_up = optional(b_up_, "b_up");
  const int code = check(x, "x");
  const c10::Device dev = x.device();
  if (x.dim() < 1) throw py::value_error("x must have at least one dimension");
  const int64_t width = x.size(-1);
  const struct {
    const Tensor& t;
    const char* name;
    int64_t dim;
  } others[] = {{w_gate, "w_gate", 2}, {w_up, "w_up", 2}, {b_gate, "b_gate", 1}, {b_up, "b_up", 1}};
  for (const auto& o : others) {
    if (!o.t.defined()) continue;
    if (check(o.t, o.name) != code) throw py::type_error(std::string(o.name) + " must have x's dtype");
    check_device(o.t, dev, o.name);
    if (o.t.dim() != o.dim || o.t.size(0) != w_gate.size(0) || (o.dim == 2 && o.t.size(1) != width))
      throw py::value_error(std::string(o.name) + (o.dim == 2 ? " must be [hidden, width], with x's width and w_gate's hidden"
                                                              : " must have one value for each of the hidden"));
  }
  const int64_t hidden = w_gate.size(0), most = 1 << 20;
  if (width < 1 || width > most || hidden < 1 || hidden > most)
    throw py::value_error("width and hidden must be 1 to " + std::to_string(most));
  const c10::DeviceGuard guard(dev);
  const bool wants = wants_gradient({&x, &w_gate, &w_up, &b_gate, &b_up});
  torch::autograd::edge_list edges;
  if (wants) {
    edges = edges_of({&x, &w_gate, &w_up, &b_gate, &b_up});
    check_capture(edges, dev, "gated_linear");
  }
  const ssim_gated_linear_inputs in = gated_inputs(x, w_gate, w_up, b_gate, b_up, act);
  auto sizes = x.sizes().vec();
  sizes.back() = hidden;
  Tensor out = fresh(sizes, x.scalar_type(), dev), g, u;
  if (wants) {
    const int64_t n = (int64_t)ssim_gated_linear_saved_elements(&in);
    g = fresh({n}, at::kFloat, dev);
    u = fresh({n}, at::kFloat, dev);
  }
  const size_t bytes = ssim_gated_linear_workspace_bytes(&in);
  const c10::DataPtr ws = bytes ? scratch(bytes) : c10::DataPtr();
  const int rc = ssim_gated_linear_forward(&in, out.data_ptr(), wants ? g.data_ptr<float>() : nullptr,
                                           wants ? u.data_ptr<float>() : nullptr, ws.get(), stream_of(dev));
  if (rc != SSIM_OK) raise(rc, "ssim_gated_linear_forward");
  if (wants) {
    std::shared_ptr<GatedLinearBackward> node(new GatedLinearBackward(), torch::autograd::deleteNode);
    const Tensor* tensors[] = {&x, &w_gate, &w_up, &b_gate, &b_up, &g, &u};
    for (int n = 0; n < GatedLinearBackward::kTensors; ++n)
      if (tensors[n]->defined()) node->saved[n] = SavedVariable(*tensors[n], false);
    node->act = act;
    node->set_next_edges(std::move(edges));
    torch::autograd::set_history(out, node);
  }
  return out;
}

}  // namespace

void add_block(py::module_& m) {
  m.def("rotary", &rotary);
  m.def("attention", &attention);
  m.def("gated_linear", &gated_linear);
}

}  // namespace ssim_bind
