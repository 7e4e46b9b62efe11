// The torch half of gradient clipping (precision_optimizer_state_amd.grads), of linear
// cross entropy and of the gated block (precision_optimizer_state_amd.nn): host C++
// that turns torch tensors into the arguments of the C ABI (include/foamd.h, which
// defines what is computed) and records the autograd graph.  It launches nothing
// itself.  It is C++ for the host's time: a list of 148 gradients is marshalled in
// microseconds.
#define FO_OPERATORS "operators of this extension"

#include "fo_torch.hpp"

#include <ATen/MemoryOverlap.h>

#include <algorithm>

namespace {

// A workspace of the current stream's: at least one byte, so that it has an address.
struct Workspace {
  Tensor held;
  int64_t bytes = 0;

  Workspace(int64_t n, const at::TensorOptions& like)
      : held(at::empty({std::max<int64_t>(n, 1)}, like.dtype(at::kByte))), bytes(n) {}
  void* ptr() const { return held.data_ptr(); }
};

// What a backward pass needs besides tensors.
struct Saved : torch::CustomClassHolder {
  int64_t ignore_index = 0;
  double smoothing = 0.0;
  int32_t which = 0;                      // the reduction, or the activation
};
void put(AutogradContext* ctx, int64_t ignore_index, double smoothing, int32_t which) {
  auto s = c10::make_intrusive<Saved>();
  s->ignore_index = ignore_index;
  s->smoothing = smoothing;
  s->which = which;
  ctx->saved_data["args"] = at::IValue::make_capsule(std::move(s));
}
c10::intrusive_ptr<Saved> saved(AutogradContext* ctx) {
  return c10::static_intrusive_pointer_cast<Saved>(ctx->saved_data["args"].toCapsule());
}

// x's leading dimensions with another last one
std::vector<int64_t> with_last(const Tensor& x, int64_t last) {
  std::vector<int64_t> s = x.sizes().vec();
  s.back() = last;
  return s;
}

void check_weight(const char* name, const Tensor& w, const Tensor& x) {
  TORCH_CHECK_VALUE(w.dim() == 2 && w.size(1) == x.size(-1) && w.size(0) > 0, name, " has shape ", sizes(w), ", not [n, ",
                    x.size(-1), "] with n of at least 1");
  TORCH_CHECK_VALUE(w.scalar_type() == x.scalar_type(), name, " is ", w.dtype(), " and x ", x.dtype(), ": they must agree");
  check_device(w);
}

void check_x(const Tensor& x) {
  TORCH_CHECK_VALUE(x.dim() > 0 && x.size(-1) > 0, "x needs a last dimension of at least one element, got shape ", sizes(x));
  check_device(x);
  dtype_of(x);
}

// ---------------------------------------------------------------------------
// linear cross entropy
// ---------------------------------------------------------------------------
struct LossArgs {
  Rows x, weight;
  Tensor target;
  fo_loss a = {};

  LossArgs(const Tensor& x_any, const Tensor& weight_any, const Tensor& target_any, int64_t ignore_index, int32_t reduction,
           double smoothing)
      : x(x_any), weight(weight_any), target(packed(target_any)) {
    a.x = x.ptr;
    a.weight = weight.ptr;
    a.target = static_cast<const int64_t*>(target.data_ptr());
    a.rows = x.rows;
    a.cols = x.cols;
    a.vocab = weight.rows;
    a.x_ld = x.ld;
    a.weight_ld = weight.ld;
    a.ignore_index = ignore_index;
    a.smoothing = smoothing;
    a.dtype = dtype_of(x.held);
    a.reduction = reduction;
  }
};

// `lse`: a row of log sums of exponentials and, where a backward pass will want them, one
// of what their rounding left
struct LossOut { Tensor loss, lse, count; };

void check_loss(const Tensor& x, const Tensor& weight, const Tensor& target) {
  check_x(x);
  check_weight("weight", weight, x);
  TORCH_CHECK_VALUE(target.scalar_type() == at::kLong, "target must be int64, got ", target.dtype());
  TORCH_CHECK_VALUE(target.sizes() == x.sizes().slice(0, x.dim() - 1), "target has shape ", sizes(target),
                    ", not x's without its last dimension (x has ", sizes(x), ")");
  check_device(target);
}

LossOut loss_forward(const Tensor& x, const Tensor& weight, const Tensor& target, int64_t ignore_index, int32_t reduction,
                     double smoothing, bool keep) {
  LossArgs l(x, weight, target, ignore_index, reduction, smoothing);
  const auto f32 = x.options().dtype(at::kFloat);
  LossOut o;
  o.loss = reduction == FO_LOSS_NONE ? at::empty(target.sizes(), f32) : at::empty({}, f32);
  o.lse = at::empty({keep ? 2 : 1, l.a.rows}, f32);
  if (reduction != FO_LOSS_NONE) o.count = at::empty({}, f32);
  l.a.loss = static_cast<float*>(o.loss.data_ptr());
  l.a.lse = static_cast<float*>(o.lse.data_ptr());
  l.a.count = static_cast<float*>(address(o.count));
  int64_t bytes = 0;
  check(fo_loss_forward_workspace(&l.a, &bytes));
  const Workspace ws(bytes, x.options());
  l.a.workspace = ws.ptr();
  l.a.workspace_bytes = ws.bytes;
  check(keep ? fo_loss_forward_rest(&l.a, l.a.lse + l.a.rows, current_stream()) : fo_loss_forward(&l.a, current_stream()));
  return o;
}

struct Loss : torch::autograd::Function<Loss> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& weight, const Tensor& target,
                        int64_t ignore_index, int64_t reduction, double smoothing) {
    LossOut o = loss_forward(x, weight, target, ignore_index, static_cast<int32_t>(reduction), smoothing, true);
    ctx->save_for_backward({x, weight, target, o.lse, o.count});
    put(ctx, ignore_index, smoothing, static_cast<int32_t>(reduction));
    ctx->set_materialize_grads(false);
    return o.loss;
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    variable_list out(6);
    if (!grads[0].defined()) return out;
    const variable_list back = ctx->get_saved_variables();
    const Tensor &x = back[0], &weight = back[1], &target = back[2];
    const auto args = saved(ctx);
    check_plain({&grads[0]});
    check_loss(x, weight, target);
    LossArgs l(x, weight, target, args->ignore_index, args->which, args->smoothing);
    const Tensor lse = kept(back[3], {2, l.a.rows}), count = args->which == FO_LOSS_MEAN ? kept(back[4], {}) : Tensor();
    TORCH_CHECK_VALUE(grads[0].sizes() == (args->which == FO_LOSS_NONE ? target.sizes() : at::IntArrayRef()),
                      "the loss's gradient has shape ", sizes(grads[0]));
    const Tensor dloss = packed(grads[0]);
    if (ctx->needs_input_grad(0)) out[0] = empty_like_shape(x);
    if (ctx->needs_input_grad(1)) out[1] = empty_like_shape(weight);
    l.a.lse = static_cast<float*>(lse.data_ptr());
    l.a.count = static_cast<float*>(address(count));
    l.a.dloss = static_cast<const float*>(dloss.data_ptr());
    l.a.dloss_ld = 1;
    l.a.dx = address(out[0]);
    l.a.dweight = address(out[1]);
    int64_t bytes = 0;
    check(fo_loss_backward_workspace(&l.a, &bytes));
    const Workspace ws(bytes, x.options());
    l.a.workspace = ws.ptr();
    l.a.workspace_bytes = ws.bytes;
    check(fo_loss_backward_rest(&l.a, l.a.lse + l.a.rows, current_stream()));
    return once(std::move(out));
  }
};

Tensor linear_cross_entropy(const Tensor& x, const Tensor& weight, const Tensor& target, int64_t ignore_index,
                            int64_t reduction, double smoothing) {
  check_plain({&x, &weight});
  check_loss(x, weight, target);
  if (at::GradMode::is_enabled() && (x.requires_grad() || weight.requires_grad())) {
    check_capture({&x, &weight});
    return Loss::apply(x, weight, target, ignore_index, reduction, smoothing);
  }
  return loss_forward(x, weight, target, ignore_index, static_cast<int32_t>(reduction), smoothing, false).loss;
}

// ---------------------------------------------------------------------------
// the gated block
// ---------------------------------------------------------------------------
struct GatedArgs {
  Rows x, gate, up;
  fo_gated a = {};

  GatedArgs(const Tensor& x_any, const Tensor& gate_any, const Tensor& up_any, int32_t activation)
      : x(x_any), gate(gate_any), up(up_any) {
    a.x = x.ptr;
    a.gate = gate.ptr;
    a.up = up.ptr;
    a.rows = x.rows;
    a.cols = x.cols;
    a.features = gate.rows;
    a.x_ld = x.ld;
    a.gate_ld = gate.ld;
    a.up_ld = up.ld;
    a.dtype = dtype_of(x.held);
    a.activation = activation;
  }
};

struct GatedOut { Tensor y, g, u; };

void check_gated(const Tensor& x, const Tensor& gate, const Tensor& up) {
  check_x(x);
  check_weight("gate_weight", gate, x);
  check_weight("up_weight", up, x);
  TORCH_CHECK_VALUE(gate.sizes() == up.sizes(), "gate_weight has shape ", sizes(gate), " and up_weight ", sizes(up),
                    ": they must agree");
}

GatedOut gated_forward(const Tensor& x, const Tensor& gate, const Tensor& up, int32_t activation, bool keep) {
  GatedArgs l(x, gate, up, activation);
  GatedOut o;
  o.y = at::empty(with_last(x, gate.size(0)), x.options());
  if (keep) {
    o.g = at::empty({l.a.rows, l.a.features}, x.options().dtype(at::kFloat));
    o.u = at::empty_like(o.g);
  }
  l.a.y = o.y.data_ptr();
  l.a.g = static_cast<float*>(address(o.g));
  l.a.u = static_cast<float*>(address(o.u));
  int64_t bytes = 0;
  check(fo_gated_forward_workspace(&l.a, &bytes));
  const Workspace ws(bytes, x.options());
  l.a.workspace = ws.ptr();
  l.a.workspace_bytes = ws.bytes;
  check(fo_gated_forward(&l.a, current_stream()));
  return o;
}

struct Gated : torch::autograd::Function<Gated> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& gate, const Tensor& up, int64_t activation) {
    GatedOut o = gated_forward(x, gate, up, static_cast<int32_t>(activation), true);
    ctx->save_for_backward({x, gate, up, o.g, o.u});
    put(ctx, 0, 0.0, static_cast<int32_t>(activation));
    ctx->set_materialize_grads(false);
    return o.y;
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    variable_list out(4);
    if (!grads[0].defined()) return out;
    const variable_list back = ctx->get_saved_variables();
    const Tensor &x = back[0], &gate = back[1], &up = back[2];
    check_plain({&grads[0]});
    check_gated(x, gate, up);
    GatedArgs l(x, gate, up, saved(ctx)->which);
    const Tensor g = kept(back[3], {l.a.rows, l.a.features}), u = kept(back[4], {l.a.rows, l.a.features});
    const Rows dy(grads[0]);
    TORCH_CHECK_VALUE(dy.rows == l.a.rows && dy.cols == l.a.features && grads[0].scalar_type() == x.scalar_type(),
                      "the gradient is ", sizes(grads[0]), " of ", grads[0].dtype(), ", x ", sizes(x), " of ", x.dtype());
    if (ctx->needs_input_grad(0)) out[0] = empty_like_shape(x);
    if (ctx->needs_input_grad(1)) out[1] = empty_like_shape(gate);
    if (ctx->needs_input_grad(2)) out[2] = empty_like_shape(up);
    l.a.g = static_cast<float*>(g.data_ptr());
    l.a.u = static_cast<float*>(u.data_ptr());
    l.a.dy = dy.ptr;
    l.a.dy_ld = dy.ld;
    l.a.dx = address(out[0]);
    l.a.dgate = address(out[1]);
    l.a.dup = address(out[2]);
    int64_t bytes = 0;
    check(fo_gated_backward_workspace(&l.a, &bytes));
    const Workspace ws(bytes, x.options());
    l.a.workspace = ws.ptr();
    l.a.workspace_bytes = ws.bytes;
    check(fo_gated_backward(&l.a, current_stream()));
    return once(std::move(out));
  }
};

Tensor gated_linear(const Tensor& x, const Tensor& gate, const Tensor& up, int64_t activation) {
  check_plain({&x, &gate, &up});
  check_gated(x, gate, up);
  if (at::GradMode::is_enabled() && (x.requires_grad() || gate.requires_grad() || up.requires_grad())) {
    check_capture({&x, &gate, &up});
    return Gated::apply(x, gate, up, activation);
  }
  return gated_forward(x, gate, up, static_cast<int32_t>(activation), false).y;
}

// ---------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------
// (check_device asks for the current device; a list's tensors ask once)
void check_grad(const Tensor& g, c10::DeviceIndex device) {
  TORCH_CHECK_VALUE(g.defined() && g.layout() == at::kStrided, "gradients must be dense tensors");
  if (!g.is_cuda() || g.device().index() != device) check_device(g);
  dtype_of(g);
  TORCH_CHECK_NOT_IMPLEMENTED(!g._fw_grad(/*level=*/0).defined(), "the " FO_OPERATORS " have no forward-mode derivatives");
}
// The norm, whose derivatives by tensors of a graph are not provided.
Tensor as_result(const Tensor& norm, const std::vector<Tensor>& grads) {
  bool graph = false;
  for (const Tensor& g : grads) graph |= g.requires_grad();
  if (!graph) return norm;
  return without_derivative({norm}, "the norm of gradients has no derivative")[0];
}
// The current device, or that of a tensor off the GPU, whose check then says so.
c10::DeviceIndex device_of(const std::vector<Tensor>& list) {
  return list.empty() || !list[0].defined() || !list[0].is_cuda() ? c10::DeviceIndex(-1) : c10::hip::current_device();
}

// Whether a tensor's elements are one stretch of memory, in whatever order.
bool flat(const Tensor& t) { return !t.is_neg() && t.is_non_overlapping_and_dense(); }

at::TensorOptions on_current_device(at::ScalarType dtype) {
  return at::TensorOptions().dtype(dtype).device(at::kCUDA, c10::hip::current_device());
}

Workspace grad_workspace() {
  int64_t bytes = 0;
  check(fo_grad_workspace(&bytes));
  return Workspace(bytes, on_current_device(at::kByte));
}

Tensor grad_norm(const std::vector<Tensor>& grads, int64_t order) {
  check_plain({});
  std::vector<fo_grad> list(grads.size());
  std::vector<Tensor> held;
  const auto device = device_of(grads);
  for (size_t i = 0; i < grads.size(); ++i) {
    const Tensor& g = grads[i];
    check_grad(g, device);
    const Tensor* t = &g;
    if (!flat(g)) t = &held.emplace_back(resolved(g.detach()).contiguous());
    list[i] = {t->data_ptr(), nullptr, t->numel(), dtype_of(g), 0};
    // (held may move its tensors as it grows; their addresses on the GPU stay)
  }
  const Tensor norm = at::empty({}, on_current_device(at::kFloat));
  const Workspace ws = grad_workspace();
  check(fo_grad_norm(list.data(), static_cast<int32_t>(list.size()), static_cast<int32_t>(order),
                     static_cast<float*>(norm.data_ptr()), ws.ptr(), ws.bytes, current_stream()));
  return as_result(norm, grads);
}

// Clips `grads` into `outs` (the same tensors: in place); the norm.
Tensor clip(const std::vector<Tensor>& grads, const std::vector<Tensor>& outs, double max_norm, int64_t order) {
  check_plain({});
  TORCH_CHECK_VALUE(grads.size() == outs.size(), grads.size(), " gradients are clipped into ", outs.size(), " tensors");
  at::NoGradGuard guard;
  std::vector<fo_grad> list(grads.size());
  std::vector<Tensor> held;
  std::vector<std::pair<Tensor, Tensor>> back;          // copies to write back
  const auto device = device_of(grads);
  for (size_t i = 0; i < grads.size(); ++i) {
    const Tensor &g = grads[i], &o = outs[i];
    check_grad(g, device);
    if (!g.is_same(o)) check_grad(o, device);
    TORCH_CHECK_VALUE(g.sizes() == o.sizes(), "a gradient of shape ", sizes(g), " is clipped into ", sizes(o));
    const bool in_place = g.is_same(o);
    const bool direct = flat(g) && flat(o) && g.strides() == o.strides();
    Tensor from = g, to = o;
    if (!direct) {
      // through packed copies; in place, the copy is clipped and written back (what cannot be
      // written back is refused here, before anything is written)
      at::assert_no_internal_overlap(o);
      from = flat(g) && g.is_contiguous() ? g : resolved(g.detach()).clone(at::MemoryFormat::Contiguous);
      to = in_place ? from : flat(o) && o.is_contiguous() ? o : at::empty(o.sizes(), o.options());
      held.push_back(from);
      if (!to.is_same(o)) back.emplace_back(o, to);
    }
    list[i] = {from.data_ptr(), to.data_ptr(), from.numel(), dtype_of(from), dtype_of(to)};
  }
  // (the library refuses a tensor that is listed twice; copies hide it)
  std::sort(back.begin(), back.end(), [](const auto& a, const auto& b) { return a.first.data_ptr() < b.first.data_ptr(); });
  for (size_t i = 1; i < back.size(); ++i) {
    const Tensor &a = back[i - 1].first, &b = back[i].first;
    TORCH_CHECK_VALUE(a.numel() == 0 || a.data_ptr() != b.data_ptr() || a.sizes() != b.sizes() || a.strides() != b.strides(),
                      "a tensor is listed twice");
  }
  const Tensor norm = at::empty({}, on_current_device(at::kFloat));
  const Workspace ws = grad_workspace();
  check(fo_grad_clip(list.data(), static_cast<int32_t>(list.size()), static_cast<int32_t>(order), max_norm,
                     static_cast<float*>(norm.data_ptr()), ws.ptr(), ws.bytes, current_stream()));
  {
    // (as the kernels write the others: versions follow below, and inference tensors have none)
    at::AutoDispatchBelowADInplaceOrView below;
    for (auto& [o, t] : back) o.copy_(t);
  }
  // a graph that saved one of these tensors must not be run on what it holds now
  for (const Tensor& o : outs)
    if (!o.is_inference()) o.unsafeGetTensorImpl()->bump_version();
  return norm;
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.doc() = "gradient clipping, linear cross entropy and the gated block: autograd and marshalling (host code)";
  m.def("linear_cross_entropy", &linear_cross_entropy, py::arg("x"), py::arg("weight"), py::arg("target"),
        py::arg("ignore_index"), py::arg("reduction"), py::arg("smoothing"));
  m.def("gated_linear", &gated_linear, py::arg("x"), py::arg("gate_weight"), py::arg("up_weight"), py::arg("activation"));
  m.def("grad_norm", &grad_norm, py::arg("grads"), py::arg("order"));
  m.def("clip", &clip, py::arg("grads"), py::arg("outs"), py::arg("max_norm"), py::arg("order"));
  define_error(m);
}
