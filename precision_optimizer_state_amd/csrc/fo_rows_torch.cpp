// The autograd half of the row operators (precision_optimizer_state_amd.nn):
// host C++ that turns torch tensors into the arguments of the C ABI
// (include/foamd.h, which defines what is computed) and records the autograd
// graph.  It does no arithmetic and launches nothing itself.  It is C++ because
// a small call costs more on the host than on the GPU: a forward and backward
// pass through a Python autograd.Function took 140-230 us of host time, whatever
// the size.
#define FO_OPERATORS "row operators"

#include <ATen/CPUGeneratorImpl.h>
#include <ATen/SavedTensorHooks.h>

#include "fo_torch.hpp"

namespace {

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
    const Tensor state = ctx->get_saved_variables()[0];
    check_key(Saved::get(ctx)->key, state);
    return once({drop(grads[0], Saved::get(ctx)->key, state), Tensor(), Tensor()});
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
void check_row(const Tensor& x) {
  TORCH_CHECK_VALUE(x.dim() > 0 && x.size(-1) > 0,
                    "a norm needs a last dimension of at least one element, got shape ", sizes(x));
  check_device(x);
  dtype_of(x);
}
void check_param(const char* name, const Tensor& t, const Tensor& x) {
  if (!t.defined()) return;
  TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == x.size(-1), name, " has shape ", sizes(t), ", not [", x.size(-1), "]");
  check_device(t);
  dtype_of(t);
}

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
    const Tensor &h = saved[0], &weight = saved[1], &state = saved[3];
    const auto args = Saved::get(ctx);
    const Key& key = args->key;
    const bool join = grads.size() == 2;
    const Tensor dy = grads.back(), dh = join ? grads[0] : Tensor();
    check_plain({&dy, &dh});
    check_key(key, state);
    check_row(h);
    check_param("weight", weight, h);
    TORCH_CHECK_VALUE(!weight.defined() || args->bias_dtype == at::ScalarType::Undefined ||
                          weight.scalar_type() == args->bias_dtype,
                      "weight is ", weight.dtype(), " and bias ", args->bias_dtype, ": they must agree");
    for (const Tensor& g : {dy, dh})
      TORCH_CHECK_VALUE(!g.defined() || (g.sizes() == h.sizes() && g.scalar_type() == h.scalar_type()), "a gradient is ",
                        sizes(g), " of ", g.dtype(), ", the rows ", sizes(h), " of ", h.dtype());
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
    const Tensor stats = kept(saved[2], {args->kind == FO_LAYER_NORM ? 2 : 1, rh.rows});
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
  check_row(x);
  bool grad = x.requires_grad();
  for (const auto& [name, t] : {std::pair<const char*, const Tensor&>{"weight", weight}, {"bias", bias}}) {
    check_param(name, t, x);
    grad |= t.defined() && t.requires_grad();
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
  define_error(m);
}
