// The autograd half of the row operators (precision_optimizer_state_amd.nn):
// host C++ that turns torch tensors into the arguments of the C ABI
// (include/foamd.h, which defines what is computed) and records the autograd
// graph.  It does no arithmetic and launches nothing itself.  It is C++ because
// a small call costs more on the host than on the GPU: a forward and backward
// pass through a Python autograd.Function took 140-230 us of host time, whatever
// the size.
#include <ATen/CPUGeneratorImpl.h>
#include <ATen/SavedTensorHooks.h>
#include <ATen/TracerMode.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/graph_task.h>
#include <torch/extension.h>

#include <cstdint>
#include <optional>
#include <string>

#include "../../include/foamd.h"

namespace py = pybind11;
using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
// An absent input of an autograd function has to be an empty optional (it then
// takes no place among the function's inputs); elsewhere it is an undefined tensor.
using MaybeTensor = std::optional<Tensor>;

namespace {

Tensor value(const MaybeTensor& t) { return t.value_or(Tensor()); }

// A failing library call; becomes precision_optimizer_state_amd.FoError.
struct LibraryError : std::runtime_error {
  LibraryError(int c, const std::string& m) : std::runtime_error("[" + std::to_string(c) + "] " + m), code(c), message(m) {}
  int code;
  std::string message;
};

void check(int rc) {
  if (rc != FO_OK) throw LibraryError(rc, fo_last_error());
}

std::string sizes(const Tensor& t) {
  std::ostringstream s;
  s << t.sizes();
  return s.str();
}

int dtype_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return FO_BF16;
    case at::kHalf: return FO_FP16;
    case at::kFloat: return FO_F32;
    default: TORCH_CHECK_VALUE(false, "tensors of ", t.dtype(), " are not supported (bfloat16, float16 or float32)");
  }
}

// The library launches on the current device and dereferences addresses there.
void check_device(const Tensor& t) {
  TORCH_CHECK_VALUE(t.is_cuda(), "tensors passed to the library must live on the GPU (got one on ", t.device(), ")");
  const auto dev = c10::hip::current_device();
  TORCH_CHECK_VALUE(t.device().index() == dev, "a tensor lives on ", t.device(), ", but the current device is cuda:",
                    static_cast<int>(dev));
}

// A tracer (make_fx, torch.jit.trace) sees the outputs' allocations and no launch.
bool traced() {
  using Modes = c10::impl::TorchDispatchModeTLS;
  return at::tracer::impl::is_dispatch_enabled() || c10::impl::tls_is_dispatch_key_included(c10::DispatchKey::PreDispatch) ||
         (Modes::any_modes_set() && Modes::get_mode(c10::impl::TorchDispatchModeKey::PROXY));
}

// Kernels are launched on addresses: a tangent that rides on an input would be
// left out of what comes back, no derivative instead of an error, and a trace
// would replay as memory that nothing has written.
void check_plain(std::initializer_list<const Tensor*> inputs) {
  TORCH_CHECK_NOT_IMPLEMENTED(!traced(), "the row operators cannot be traced (make_fx, torch.jit.trace)");
  for (const Tensor* t : inputs)
    TORCH_CHECK_NOT_IMPLEMENTED(!t->defined() || !t->_fw_grad(/*level=*/0).defined(),
                                "the row operators have no forward-mode derivatives");
}

void* current_stream() { return c10::hip::getCurrentHIPStream().stream(); }

// Under capture, the gradient of an input whose place in the autograd graph was
// made on the default stream (a leaf that an eager graph, still alive, has used
// too) would make that stream wait for the capturing one.  The runtime forbids
// it, and the autograd engine ends the process when it happens in the captured
// backward pass, so the forward call is refused.
void check_capture(std::initializer_list<const Tensor*> inputs) {
  if (c10::hip::currentStreamCaptureStatusMayInitCtx() == c10::hip::CaptureStatus::None) return;
  for (const Tensor* t : inputs) {
    if (!t->defined() || !t->requires_grad()) continue;
    const auto made_on = torch::autograd::impl::gradient_edge(*t).function->stream();
    TORCH_CHECK(!made_on || made_on->id() != 0,
                "this call is captured into a graph, but an input's gradient belongs to an autograd graph made on the "
                "default stream: release that graph first, or capture with inputs detached from it");
  }
}

// A view that torch negates when it reads it (the imaginary part of a conjugate)
// holds the other sign in memory.
Tensor resolved(const Tensor& t) { return t.is_neg() ? t.resolve_neg() : t; }

// A tensor as a matrix: cols its last dimension, rows everything before.  The
// tensor's own memory where its rows are consecutive elements at a constant
// distance, else a packed copy (held here).
struct Rows {
  Tensor held;
  void* ptr;
  int64_t rows, cols, ld;

  explicit Rows(const Tensor& any) : held(resolved(any)) {
    const Tensor t = held;
    cols = t.dim() ? t.size(-1) : 1;
    rows = cols ? t.numel() / cols : 0;
    ld = cols;
    bool packed = t.is_contiguous();
    if (!packed && t.numel() && (t.stride(-1) == 1 || cols == 1)) {
      // strides of the leading dimensions of more than one element, from the
      // inside: each must step over all the rows of the ones before it
      int64_t step = -1, inner = 1;
      bool even = true;
      for (int64_t i = t.dim() - 2; i >= 0; --i) {
        const int64_t n = t.size(i);
        if (n == 1) continue;
        if (step < 0) step = t.stride(i);
        else even &= t.stride(i) == step * inner;
        inner *= n;
      }
      if (even) {
        ld = step < 0 ? cols : step;
        packed = true;
      }
    }
    if (!packed) held = t.contiguous();
    ptr = held.data_ptr();
  }
};

void* address(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

Tensor packed(const Tensor& t) { return t.defined() ? resolved(t).contiguous() : t; }

Tensor empty_like_shape(const Tensor& t) { return at::empty(t.sizes(), t.options()); }

// seed, offset and drop probability of one call, and the tensor added to them
struct Key {
  double p = 0.0;
  uint64_t seed = 0, offset = 0;

  fo_dropout_key with(const Tensor& state) const {
    return {p, seed, offset, state.defined() ? reinterpret_cast<const uint64_t*>(state.data_ptr()) : nullptr};
  }
};

// What a backward pass needs besides tensors, kept as one entry of the context.
struct Saved : torch::CustomClassHolder {
  Key key;
  int32_t kind = 0;
  at::ScalarType bias_dtype = at::ScalarType::Undefined;

  static void put(AutogradContext* ctx, const Key& key, int32_t kind = 0,
                  at::ScalarType bias_dtype = at::ScalarType::Undefined) {
    auto s = c10::make_intrusive<Saved>();
    s->key = key;
    s->kind = kind;
    s->bias_dtype = bias_dtype;
    ctx->saved_data["args"] = at::IValue::make_capsule(std::move(s));
  }
  static c10::intrusive_ptr<Saved> get(AutogradContext* ctx) {
    return c10::static_intrusive_pointer_cast<Saved>(ctx->saved_data["args"].toCapsule());
  }
};

void check_key(const Key& k, const Tensor& state) {
  TORCH_CHECK_VALUE(k.p >= 0.0 && k.p <= 1.0, "the drop probability must lie in [0, 1], got ", k.p);
  if (!state.defined()) return;
  TORCH_CHECK_VALUE(state.scalar_type() == at::kLong && state.numel() == 2 && state.is_contiguous(),
                    "the dropout state must hold 2 int64");
  TORCH_CHECK_VALUE(!state.is_neg(), "the dropout state is a negated view");
  check_device(state);
}

// Gradients carry no graph of their own: a second differentiation through them
// fails instead of leaving this operator's part out.
variable_list once(variable_list grads) {
  if (!at::GradMode::is_enabled()) return grads;
  variable_list defined;
  for (const auto& g : grads)
    if (g.defined()) defined.push_back(g.detach());
  if (defined.empty()) return grads;
  for (auto& g : defined) g.requires_grad_(true);
  const auto error = std::make_shared<torch::autograd::DelayedError>("the row operators have no second derivatives",
                                                                     static_cast<int64_t>(defined.size()));
  const variable_list out = (*error)(std::move(defined));
  size_t i = 0;
  for (auto& g : grads)
    if (g.defined()) g = out[i++];
  return grads;
}

// ---------------------------------------------------------------------------
// dropout
// ---------------------------------------------------------------------------
Tensor drop(const Tensor& x, const Key& key, const Tensor& state) {
  Tensor y = empty_like_shape(x);
  if (!x.numel()) return y;
  const Rows r(x);
  const fo_dropout_key k = key.with(state);
  check(fo_dropout(r.ptr, r.ld, y.data_ptr(), r.rows, r.cols, dtype_of(x), &k, current_stream()));
  return y;
}

struct Dropout : torch::autograd::Function<Dropout> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Key& key, const MaybeTensor& state) {
    ctx->save_for_backward({value(state)});
    Saved::put(ctx, key);
    return drop(x, key, value(state));
  }
  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    check_plain({&grads[0]});
    return once({drop(grads[0], Saved::get(ctx)->key, ctx->get_saved_variables()[0]), Tensor(), Tensor()});
  }
};

Tensor dropout(const Tensor& x, double p, uint64_t seed, uint64_t offset, const MaybeTensor& state) {
  const Key key{p, seed, offset};
  check_key(key, value(state));
  if (p == 0.0) return x;
  check_plain({&x});
  check_device(x);
  dtype_of(x);
  if (at::GradMode::is_enabled() && x.requires_grad()) {
    check_capture({&x});
    return Dropout::apply(x, key, state);
  }
  return drop(x, key, value(state));
}

// ---------------------------------------------------------------------------
// norms
// ---------------------------------------------------------------------------
struct Forward {
  Tensor h, y, stats;     // stats: rstd of every row, then (layer norm) the means
};

Forward norm_forward(const Tensor& x, const Tensor& residual, const Tensor& weight, const Tensor& bias, double eps,
                     int kind, const Key& key, const Tensor& state, bool stats) {
  const Rows r(x);
  std::optional<Rows> res;
  if (residual.defined()) res.emplace(residual);
  const Tensor w = packed(weight), b = packed(bias);
  const Tensor& param = w.defined() ? w : b;
  Forward f;
  f.y = empty_like_shape(x);
  if (res) f.h = empty_like_shape(x);
  if (stats) f.stats = at::empty({kind == FO_LAYER_NORM ? 2 : 1, r.rows}, x.options().dtype(at::kFloat));
  fo_norm_fwd a = {};
  a.x = r.ptr;
  a.residual = res ? res->ptr : nullptr;
  a.weight = address(w);
  a.bias = address(b);
  a.h = address(f.h);
  a.y = f.y.data_ptr();
  a.rstd = static_cast<float*>(address(f.stats));
  a.mean = a.rstd && kind == FO_LAYER_NORM ? a.rstd + r.rows : nullptr;
  a.rows = r.rows;
  a.cols = r.cols;
  a.x_ld = r.ld;
  a.residual_ld = res ? res->ld : 0;
  a.eps = eps;
  a.drop = key.with(state);
  a.dtype = dtype_of(x);
  a.wdtype = param.defined() ? dtype_of(param) : a.dtype;
  a.kind = kind;
  check(fo_norm_forward(&a, current_stream()));
  return f;
}

struct Norm : torch::autograd::Function<Norm> {
  static variable_list forward(AutogradContext* ctx, const Tensor& x, const MaybeTensor& residual,
                               const MaybeTensor& weight, const MaybeTensor& bias, double eps, int64_t kind,
                               const Key& key, const MaybeTensor& state) {
    Forward f = norm_forward(x, value(residual), value(weight), value(bias), eps, static_cast<int>(kind), key,
                             value(state), true);
    // a state that no mask came from may change before the backward pass
    ctx->save_for_backward({f.h.defined() ? f.h : x, value(weight), f.stats, key.p != 0.0 ? value(state) : Tensor()});
    Saved::put(ctx, key, static_cast<int32_t>(kind), bias ? bias->scalar_type() : at::ScalarType::Undefined);
    ctx->set_materialize_grads(false);
    if (f.h.defined()) return {f.h, f.y};
    return {f.y};
  }

  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &h = saved[0], &weight = saved[1], &stats = saved[2], &state = saved[3];
    const auto args = Saved::get(ctx);
    const Key& key = args->key;
    const bool join = grads.size() == 2;
    const Tensor dy = grads.back(), dh = join ? grads[0] : Tensor();
    check_plain({&dy, &dh});
    // the inputs that were there, in the order of forward's arguments
    size_t input = 0;
    const bool need_x = ctx->needs_input_grad(input++);
    const bool need_res = join && ctx->needs_input_grad(input++);
    const bool need_w = weight.defined() && ctx->needs_input_grad(input++);
    const bool need_b = args->bias_dtype != at::ScalarType::Undefined && ctx->needs_input_grad(input++);
    variable_list out(8);
    if (!dy.defined()) {                    // only h was used: the norm has no part in it
      if (!dh.defined()) return out;
      if (need_x) out[0] = key.p != 0.0 ? drop(dh, key, state) : dh;
      if (need_res) out[1] = dh;
      return once(std::move(out));
    }
    const Rows rh(h), rdy(dy);
    std::optional<Rows> rdh;
    if (dh.defined()) rdh.emplace(dh);
    // without dropout the gradients of x and of the residual are one tensor
    Tensor d, dx, dw, db, workspace;
    if (need_res || (need_x && key.p == 0.0)) d = empty_like_shape(h);
    if (need_x && key.p != 0.0) dx = empty_like_shape(h);
    if (need_w) dw = empty_like_shape(weight);
    if (need_b) db = at::empty({rh.cols}, h.options().dtype(args->bias_dtype));
    const Tensor w = packed(weight);
    const Tensor& param = w.defined() ? w : db;
    fo_norm_bwd a = {};
    if (need_w || need_b) {
      check(fo_norm_backward_workspace(rh.rows, rh.cols, &a.workspace_bytes));
      workspace = at::empty({a.workspace_bytes}, h.options().dtype(at::kByte));
      a.workspace = workspace.data_ptr();
    }
    a.dy = rdy.ptr;
    a.dh = rdh ? rdh->ptr : nullptr;
    a.h = rh.ptr;
    a.weight = address(w);
    a.rstd = static_cast<const float*>(address(stats));
    a.mean = a.rstd && args->kind == FO_LAYER_NORM ? a.rstd + rh.rows : nullptr;
    a.d = address(d);
    a.dx = address(dx);
    a.dweight = address(dw);
    a.dbias = address(db);
    a.rows = rh.rows;
    a.cols = rh.cols;
    a.dy_ld = rdy.ld;
    a.dh_ld = rdh ? rdh->ld : 0;
    a.h_ld = rh.ld;
    a.drop = key.with(state);
    a.dtype = dtype_of(h);
    a.wdtype = param.defined() ? dtype_of(param) : a.dtype;
    a.kind = args->kind;
    check(fo_norm_backward(&a, current_stream()));
    if (need_x) out[0] = key.p != 0.0 ? dx : d;
    if (need_res) out[1] = d;
    out[2] = dw;
    out[3] = db;
    return once(std::move(out));
  }
};

// [y], or [h, y] with a residual
variable_list norm(const Tensor& x, const MaybeTensor& residual_arg, const MaybeTensor& weight_arg,
                   const MaybeTensor& bias_arg, double eps, int kind, double p, uint64_t seed, uint64_t offset,
                   const MaybeTensor& state_arg) {
  const Key key{p, seed, offset};
  const Tensor residual = value(residual_arg), weight = value(weight_arg), bias = value(bias_arg);
  const Tensor state = value(state_arg);
  check_key(key, state);
  check_plain({&x, &residual, &weight, &bias});
  TORCH_CHECK_VALUE(x.dim() > 0 && x.size(-1) > 0,
                    "a norm needs a last dimension of at least one element, got shape ", sizes(x));
  check_device(x);
  dtype_of(x);
  bool grad = x.requires_grad();
  for (const auto& [name, t] : {std::pair<const char*, const Tensor&>{"weight", weight}, {"bias", bias}}) {
    if (!t.defined()) continue;
    TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == x.size(-1), name, " has shape ", sizes(t), ", not [", x.size(-1), "]");
    check_device(t);
    dtype_of(t);
    grad |= t.requires_grad();
  }
  if (weight.defined() && bias.defined())
    TORCH_CHECK_VALUE(weight.scalar_type() == bias.scalar_type(), "weight is ", weight.dtype(), " and bias ",
                      bias.dtype(), ": they must agree");
  if (residual.defined()) {
    TORCH_CHECK_VALUE(residual.sizes() == x.sizes() && residual.scalar_type() == x.scalar_type(),
                      "the residual must be ", sizes(x), " of ", x.dtype(), ", got ", sizes(residual), " of ",
                      residual.dtype());
    check_device(residual);
    grad |= residual.requires_grad();
  }
  if (grad && at::GradMode::is_enabled()) {
    check_capture({&x, &residual, &weight, &bias});
    return Norm::apply(x, residual_arg, weight_arg, bias_arg, eps, static_cast<int64_t>(kind), key, state_arg);
  }
  Forward f = norm_forward(x, residual, weight, bias, eps, kind, key, state, false);
  if (f.h.defined()) return {f.h, f.y};
  return {f.y};
}

// ---------------------------------------------------------------------------
// recomputed forward passes
// ---------------------------------------------------------------------------
// Whether a backward pass may run the present forward code again, or is doing so:
// activation checkpointing runs a function first without gradients or under hooks
// on saved tensors, and again inside the backward pass, from the same state of
// torch's CPU generator.  For such a call, a number drawn from that generator
// (the same one both times) and whether this is inside a backward pass; None for
// any other.
std::optional<std::pair<int64_t, bool>> recomputation() {
  const bool backward = torch::autograd::get_current_graph_task_id() != -1;
  if (!backward) {
    if (c10::InferenceMode::is_enabled()) return std::nullopt;
    if (at::GradMode::is_enabled() && !at::SavedTensorDefaultHooks::get_hooks(/*ignore_is_tracing=*/true))
      return std::nullopt;
  }
  at::Generator gen = at::detail::getDefaultCPUGenerator();
  const std::lock_guard<std::mutex> lock(gen.mutex());
  const uint64_t drawn = at::check_generator<at::CPUGeneratorImpl>(gen)->random64();
  return std::pair<int64_t, bool>(static_cast<int64_t>(drawn >> 1), backward);
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.doc() = "autograd and marshalling of the row operators (host code)";
  m.def("dropout", &dropout, py::arg("x"), py::arg("p"), py::arg("seed"), py::arg("offset"), py::arg("state"));
  m.def("norm", &norm, py::arg("x"), py::arg("residual"), py::arg("weight"), py::arg("bias"), py::arg("eps"),
        py::arg("kind"), py::arg("p"), py::arg("seed"), py::arg("offset"), py::arg("state"));
  m.def("recomputation", &recomputation);
  // FoError, raised with (code, message)
  static py::object error;
  m.def("set_error", [](py::object cls) { error = std::move(cls); });
  py::register_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const LibraryError& e) {
      py::object value = error(e.code, e.message);
      PyErr_SetObject(error.ptr(), value.ptr());
    }
  });
  m.add_object("_unload", py::capsule([]() { error.release(); }));
}
