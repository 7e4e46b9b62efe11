"""Row operators of a training step with gradients: dropout, layer norm, RMS
norm, and dropout + residual sum + norm in one pass.

They run next to the optimizers of this package, which leave a model's
parameters as 16-bit theta': norm weights may be bfloat16, float16 or float32
next to activations of any of these types, and weight gradients come in the
weights' type, the one the fused steps read without a conversion.  What they
keep for the backward pass is small: a norm keeps its input (which the residual
stream holds anyway) and two floats per row, dropout keeps nothing (its mask is
a function of a seed, an offset and the element's place, and is found again).

    counter = DropoutCounter(seed=1)
    h, y = dropout_add_layer_norm(x, residual, ln.weight, ln.bias, p=0.1, **counter.next())

All arithmetic runs in the HIP library (fo_dropout, fo_norm_forward,
fo_norm_backward in include/foamd.h, which defines the formulas and the mask);
this module marshals tensors and records the autograd graph.  Tensors must live
on the current GPU; calls go to torch's current stream, allocate only through
torch and never synchronise, so they can be captured into HIP graphs.  Norms
are over the last dimension.  Inputs whose rows are not consecutive elements at
a constant distance are copied first.  Gradients of gradients are not provided.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as B


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t as (rows, cols), cols its last dimension: a view where the strides allow one."""
    if t.dim() == 0:
        return t.view(1, 1)
    cols = t.shape[-1]
    if t.stride(-1) != 1 and cols > 1:
        t = t.contiguous()
    shape = (t.numel() // cols if cols else 0, cols)
    try:
        return t.view(shape)
    except RuntimeError:
        return t.contiguous().view(shape)


def _flat(t):
    return None if t is None else t.contiguous()


def _check_p(p: float) -> float:
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"the drop probability must lie in [0, 1], got {p}")
    return float(p)


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------
def _drop(x, key):
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if x.numel():
        xr = _rows(x)
        B.fo_dropout(xr, y.view(xr.shape), key)
    return y


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, seed, offset, state):
        ctx.save_for_backward(state)
        ctx.args = (p, seed, offset)
        return _drop(x, B.dropout_key(p, seed, offset, state))

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        state, = ctx.saved_tensors
        return _drop(dy, B.dropout_key(*ctx.args, state)), None, None, None, None


def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0, state: torch.Tensor | None = None) -> torch.Tensor:
    """Zero each element of x with probability p and scale the others by
    1 / (1 - p).  The mask depends on (seed, offset), p, the element's row
    and column and the length of the last dimension; no mask is stored.
    `state`: 2 int64 on the GPU added to (seed, offset) when the kernels run
    (see DropoutCounter); they may not be changed before the backward pass.
    Dropped elements are 0 even where x is NaN or infinite.  p = 0 returns x."""
    if _check_p(p) == 0.0:
        return x
    return _Dropout.apply(x, float(p), seed, offset, state)


class DropoutCounter:
    """Seeds and offsets for dropout calls: next() gives the arguments of one
    call, a fresh offset each time.

    With `device`, it also holds a state tensor there: a captured graph keeps
    the offsets it was captured with and draws new masks after advance(), which
    must be called between replays (or at the end of the captured step), never
    between a forward pass and its backward pass.

    Code that runs a forward function again for its backward pass (activation
    checkpointing) must take the arguments from next() outside that function
    and pass them in, so that both runs find the same mask."""

    _STRIDE = 1 << 32       # offsets of one replay to those of the next

    def __init__(self, seed: int, offset: int = 0, device=None):
        self.seed, self.offset = int(seed), int(offset)
        self.state = None if device is None else torch.zeros(2, dtype=torch.int64, device=device)

    def next(self) -> dict:
        args = {"seed": self.seed, "offset": self.offset, "state": self.state}
        self.offset += 1
        return args

    def advance(self) -> None:
        if self.state is None:
            raise ValueError("advance() needs a counter with a device state")
        self.state[1:].add_(self._STRIDE)

    def state_dict(self) -> dict:
        return {"seed": self.seed, "offset": self.offset,
                "state": None if self.state is None else self.state.tolist()}

    def load_state_dict(self, sd: dict) -> None:
        if (sd["state"] is None) != (self.state is None):
            raise ValueError("one of the counters has a device state and the other has none")
        self.seed, self.offset = int(sd["seed"]), int(sd["offset"])
        if self.state is not None:
            self.state.copy_(torch.tensor(sd["state"], dtype=torch.int64))


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------
def _norm_forward(x, residual, weight, bias, eps, kind, key, stats):
    """(h or None, y, mean or None, rstd or None)."""
    xr = _rows(x)
    rows = xr.shape[0]
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    h = torch.empty_like(y) if residual is not None else None
    mean = torch.empty(rows, dtype=torch.float32, device=x.device) if stats and kind == "layer" else None
    rstd = torch.empty(rows, dtype=torch.float32, device=x.device) if stats else None
    B.fo_norm_forward(xr, y.view(xr.shape), kind, _flat(weight), _flat(bias), eps,
                      None if residual is None else _rows(residual), None if h is None else h.view(xr.shape),
                      mean, rstd, key)
    return h, y, mean, rstd


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps, kind, p, seed, offset, state):
        h, y, mean, rstd = _norm_forward(x, residual, weight, bias, eps, kind,
                                         B.dropout_key(p, seed, offset, state) if p else None, True)
        ctx.save_for_backward(x if h is None else h, weight, mean, rstd, state)
        ctx.args = (kind, p, seed, offset, None if bias is None else bias.dtype)
        ctx.set_materialize_grads(False)
        return y if h is None else (h, y)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        h, weight, mean, rstd, state = ctx.saved_tensors
        kind, p, seed, offset, bias_dtype = ctx.args
        dy, dh = grads[-1], grads[0] if len(grads) == 2 else None
        need_x, need_res, need_w, need_b = ctx.needs_input_grad[:4]
        key = B.dropout_key(p, seed, offset, state) if p else None
        rest = (None,) * 6
        if dy is None:                              # only h was used: the norm has no part in it
            if dh is None:
                return (None,) * 10
            dx = None if not need_x else _drop(dh, key) if key else dh
            return (dx, dh if need_res else None, None, None) + rest

        hr = _rows(h)

        def like_h():
            return torch.empty(h.shape, dtype=h.dtype, device=h.device)

        # without dropout the gradients of x and of the residual are one tensor
        d = like_h() if need_res or (need_x and not key) else None
        dx = like_h() if need_x and key else None
        dw = torch.empty(weight.shape, dtype=weight.dtype, device=h.device) if need_w else None
        db = torch.empty(hr.shape[1], dtype=bias_dtype, device=h.device) if need_b else None
        B.fo_norm_backward(_rows(dy), hr, rstd, kind, mean, _flat(weight), None if dh is None else _rows(dh),
                           None if d is None else d.view(hr.shape), None if dx is None else dx.view(hr.shape),
                           dw, db, drop=key)
        if need_x and not key:
            dx = d
        return (dx, d if need_res else None, dw, db) + rest


def _norm(x, residual, weight, bias, eps, kind, p, seed, offset, state):
    p = _check_p(p)
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError(f"a norm needs a last dimension of at least one element, got shape {tuple(x.shape)}")
    cols = x.shape[-1]
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None and t.shape != (cols,):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, not ({cols},)")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError(f"weight is {weight.dtype} and bias {bias.dtype}: they must agree")
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError(f"the residual must be {tuple(x.shape)} of {x.dtype}, "
                         f"got {tuple(residual.shape)} of {residual.dtype}")
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, residual, weight, bias)):
        return _Norm.apply(x, residual, weight, bias, float(eps), kind, p, seed, offset, state)
    h, y, _, _ = _norm_forward(x, residual, weight, bias, eps, kind,
                               B.dropout_key(p, seed, offset, state) if p else None, False)
    return y if h is None else (h, y)


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5) -> torch.Tensor:
    """(x - mean) / sqrt(var + eps) * weight + bias over the last dimension."""
    return _norm(x, None, weight, bias, eps, "layer", 0.0, 0, 0, None)


def rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6) -> torch.Tensor:
    """x / sqrt(mean(x^2) + eps) * weight over the last dimension."""
    return _norm(x, None, weight, None, eps, "rms", 0.0, 0, 0, None)


def dropout_add_layer_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor | None = None,
                           bias: torch.Tensor | None = None, eps: float = 1e-5, *, p: float = 0.0, seed: int = 0,
                           offset: int = 0, state: torch.Tensor | None = None):
    """(h, layer_norm(h)) with h = residual + dropout(x, p), in one pass each way.
    h is rounded to x's type, and the norm is that of the rounded h."""
    return _norm(x, residual, weight, bias, eps, "layer", p, seed, offset, state)


def dropout_add_rms_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor | None = None,
                         eps: float = 1e-6, *, p: float = 0.0, seed: int = 0, offset: int = 0,
                         state: torch.Tensor | None = None):
    """(h, rms_norm(h)) with h = residual + dropout(x, p)."""
    return _norm(x, residual, weight, None, eps, "rms", p, seed, offset, state)


# ---------------------------------------------------------------------------
# modules
# ---------------------------------------------------------------------------
def _one_dim(normalized_shape):
    shape = (normalized_shape,) if isinstance(normalized_shape, int) else tuple(normalized_shape)
    if len(shape) != 1:
        raise ValueError(f"norms are over the last dimension only, got normalized_shape {shape}")
    return shape


class FlashLayerNorm(torch.nn.LayerNorm):
    """torch.nn.LayerNorm over the last dimension, on layer_norm()."""

    def __init__(self, normalized_shape, eps: float = 1e-5, elementwise_affine: bool = True, bias: bool = True,
                 device=None, dtype=None):
        super().__init__(_one_dim(normalized_shape), eps, elementwise_affine, bias, device, dtype)

    def forward(self, x):
        if x.shape[-1:] != self.normalized_shape:
            raise ValueError(f"expected a last dimension of {self.normalized_shape[0]}, got shape {tuple(x.shape)}")
        return layer_norm(x, self.weight, self.bias, self.eps)


class FlashRMSNorm(torch.nn.RMSNorm):
    """torch.nn.RMSNorm over the last dimension, on rms_norm()."""

    def __init__(self, normalized_shape, eps: float = 1e-6, elementwise_affine: bool = True, device=None, dtype=None):
        super().__init__(_one_dim(normalized_shape), eps, elementwise_affine, device, dtype)

    def forward(self, x):
        if x.shape[-1:] != self.normalized_shape:
            raise ValueError(f"expected a last dimension of {self.normalized_shape[0]}, got shape {tuple(x.shape)}")
        return rms_norm(x, self.weight, self.eps)


class FlashDropout(torch.nn.Module):
    """torch.nn.Dropout on dropout(); `counter` (shared between modules or not)
    gives every call its mask."""

    def __init__(self, p: float, counter: DropoutCounter):
        super().__init__()
        self.p, self.counter = _check_p(p), counter

    def forward(self, x):
        if not self.training or self.p == 0.0:
            return x
        return dropout(x, self.p, **self.counter.next())

    def extra_repr(self) -> str:
        return f"p={self.p}"
