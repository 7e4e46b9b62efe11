// fo_torch.hpp -- what the torch extensions of this library share: errors, checks of
// tensors, tensors as matrices of rows, gradients that carry no graph.  An extension
// defines FO_OPERATORS, what its messages call its operators, before it includes this.
#pragma once

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

// A view that torch negates when it reads it (the imaginary part of a conjugate)
// holds the other sign in memory.
Tensor resolved(const Tensor& t) { return t.is_neg() ? t.resolve_neg() : t; }

Tensor packed(const Tensor& t) { return t.defined() ? resolved(t).contiguous() : t; }

// What a backward pass kept comes back through hooks that a program may have set
// (torch.autograd.graph.saved_tensors_hooks), as whatever these return: the kernels'
// arguments are checked again.  Float32 of a known shape, packed:
Tensor kept(const Tensor& t, at::IntArrayRef shape) {
  TORCH_CHECK_VALUE(t.defined() && t.scalar_type() == at::kFloat && t.sizes() == shape, "a tensor kept for the backward pass, ",
                    shape, " of float32, came back as ", t.defined() ? sizes(t) : "nothing");
  check_device(t);
  return packed(t);
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
  TORCH_CHECK_NOT_IMPLEMENTED(!traced(), "the " FO_OPERATORS " cannot be traced (make_fx, torch.jit.trace)");
  for (const Tensor* t : inputs)
    TORCH_CHECK_NOT_IMPLEMENTED(!t->defined() || !t->_fw_grad(/*level=*/0).defined(),
                                "the " FO_OPERATORS " have no forward-mode derivatives");
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

Tensor empty_like_shape(const Tensor& t) { return at::empty(t.sizes(), t.options()); }

// Results that carry no graph of their own: a differentiation through them fails,
// instead of leaving this operator's part out.
variable_list without_derivative(variable_list results, const char* why) {
  if (!at::GradMode::is_enabled()) return results;
  variable_list defined;
  for (const auto& g : results)
    if (g.defined()) defined.push_back(g.detach());
  if (defined.empty()) return results;
  for (auto& g : defined) g.requires_grad_(true);
  const auto error = std::make_shared<torch::autograd::DelayedError>(why, static_cast<int64_t>(defined.size()));
  const variable_list out = (*error)(std::move(defined));
  size_t i = 0;
  for (auto& g : results)
    if (g.defined()) g = out[i++];
  return results;
}
// ... the gradients of a backward pass
variable_list once(variable_list grads) {
  return without_derivative(std::move(grads), "the " FO_OPERATORS " have no second derivatives");
}

// FoError, raised with (code, message); call once in a module's definition.
void define_error(py::module_& m) {
  static py::object error;
  m.def("set_error", [](py::object cls) { error = std::move(cls); });
  py::register_local_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const LibraryError& e) {
      py::object value = error(e.code, e.message);
      PyErr_SetObject(error.ptr(), value.ptr());
    }
  });
  m.add_object("_unload", py::capsule([]() { error.release(); }));
}

}  // namespace
