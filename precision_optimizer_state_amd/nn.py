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
a host extension (csrc/fo_rows_torch.cpp) marshals tensors and records the
autograd graph.  Tensors must live on the current GPU; calls go to torch's
current stream, allocate only through torch and never synchronise, so they can
be captured into HIP graphs (a captured call refuses leaves that an eager
autograd graph, still alive, has used on the default stream: capture with
detached leaves).  Norms are over the last dimension, of at most 2^26 elements.
Inputs whose rows are not consecutive elements at a constant distance are copied
first.  Gradients of gradients and forward-mode derivatives are not provided, and
the functions cannot be traced by make_fx or torch.jit.trace: such calls are
refused.
"""

from __future__ import annotations

import collections
import copy
import importlib.util
import numbers
import os
import threading

import torch

from . import binding as B

EXT_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "fo_rows_torch.so")
_ext = None
_M64 = (1 << 64) - 1
_lock = threading.Lock()        # of all counters (one of its own would keep a counter from being copied)


def _load():
    """The host extension (autograd and marshalling), loaded once.  Raises
    ImportError when it, or the library, has not been built."""
    global _ext
    if _ext is None:
        B._load_rows()
        if not os.path.exists(EXT_PATH):
            raise ImportError(f"{EXT_PATH} is missing: build it with __graft_entry__.build()")
        spec = importlib.util.spec_from_file_location("fo_rows_torch", EXT_PATH)
        ext = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(ext)
        ext.set_error(B.FoError)
        _ext = ext
    return _ext


def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0, state: torch.Tensor | None = None) -> torch.Tensor:
    """Zero each element of x with probability p and scale the others by
    1 / (1 - p).  The mask depends on (seed, offset), p, the element's row
    and column and the length of the last dimension; no mask is stored.
    `state`: 2 int64 on the GPU added to (seed, offset) when the kernels run
    (see DropoutCounter); they may not be changed before the backward pass.
    Dropped elements are 0 even where x is NaN or infinite.  p = 0 returns x."""
    return (_ext or _load()).dropout(x, p, int(seed) & _M64, int(offset) & _M64, state)


class DropoutCounter:
    """Seeds and offsets for dropout calls: next() gives the arguments of one
    call, a fresh offset each time, also to calls from several threads.

    With `device`, it also holds a state tensor there: a captured graph keeps
    the offsets it was captured with and draws new masks after advance(), which
    must be called between replays (or at the end of the captured step), never
    between a forward pass and its backward pass.

    A forward pass that a backward pass runs again (activation checkpointing)
    finds the same arguments: next() ties those it gives out without gradients
    or under hooks on saved tensors, where a first run cannot be told from any
    other call, to one number drawn from torch's CPU generator, whose state
    torch.utils.checkpoint restores for the second run.  The same state of that
    generator then gives the same arguments again, whoever set it.  Inside a
    backward pass next() refuses a state that it has given nothing for
    (preserve_rng_state=False; a new forward pass in a hook): such code takes
    the arguments before and passes them in."""

    _STRIDE = 1 << 32       # offsets of one replay to those of the next
    _REMEMBERED = 1 << 16   # calls between a first run and its recomputation, at most

    def __init__(self, seed: int, offset: int = 0, device=None):
        self.seed, self.offset = int(seed), int(offset)
        self.state = None if device is None else torch.zeros(2, dtype=torch.int64, device=device)

    def next(self) -> dict:
        again = (_ext or _load()).recomputation()
        with _lock:
            if again is None:
                seed, offset = self._fresh()
            else:
                drawn, backward = again
                given = self.__dict__.setdefault("_given", collections.OrderedDict())
                if drawn not in given:
                    if backward:
                        raise RuntimeError(
                            "a dropout call inside a backward pass recomputes no forward call that this counter knows, so "
                            "its mask cannot be found again: keep torch's generator state (preserve_rng_state=True), or "
                            "take the arguments from next() outside the recomputed function")
                    given[drawn] = self._fresh()
                    if len(given) > self._REMEMBERED:
                        given.popitem(last=False)
                elif not backward and given[drawn] == (self.seed, self.offset):
                    self._fresh()               # a program that runs again from this state
                seed, offset = given[drawn]
        return {"seed": seed, "offset": offset, "state": self.state}

    def _fresh(self):
        offset = self.offset
        self.offset += 1
        return self.seed, offset

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
        with _lock:
            self.seed, self.offset = int(sd["seed"]), int(sd["offset"])
            self.__dict__.pop("_given", None)
        if self.state is not None:
            self.state.copy_(torch.tensor(sd["state"], dtype=torch.int64))


def _norm(x, residual, weight, bias, eps, kind, p=0.0, seed=0, offset=0, state=None):
    return (_ext or _load()).norm(x, residual, weight, bias, eps, kind, p, int(seed) & _M64, int(offset) & _M64, state)


def _join(x, residual, *args):
    if residual is None:
        raise ValueError("the fused form needs a residual")
    h, y = _norm(x, residual, *args)
    return h, y


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5) -> torch.Tensor:
    """(x - mean) / sqrt(var + eps) * weight + bias over the last dimension."""
    return _norm(x, None, weight, bias, eps, B.FO_LAYER_NORM)[0]


def rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6) -> torch.Tensor:
    """x / sqrt(mean(x^2) + eps) * weight over the last dimension."""
    return _norm(x, None, weight, None, eps, B.FO_RMS_NORM)[0]


def dropout_add_layer_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor | None = None,
                           bias: torch.Tensor | None = None, eps: float = 1e-5, *, p: float = 0.0, seed: int = 0,
                           offset: int = 0, state: torch.Tensor | None = None):
    """(h, layer_norm(h)) with h = residual + dropout(x, p), in one pass each way.
    h is rounded to x's type, and the norm is that of the rounded h."""
    return _join(x, residual, weight, bias, eps, B.FO_LAYER_NORM, p, seed, offset, state)


def dropout_add_rms_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor | None = None,
                         eps: float = 1e-6, *, p: float = 0.0, seed: int = 0, offset: int = 0,
                         state: torch.Tensor | None = None):
    """(h, rms_norm(h)) with h = residual + dropout(x, p)."""
    return _join(x, residual, weight, None, eps, B.FO_RMS_NORM, p, seed, offset, state)


# ---------------------------------------------------------------------------
# modules
# ---------------------------------------------------------------------------
def _one_dim(normalized_shape):
    shape = (normalized_shape,) if isinstance(normalized_shape, numbers.Integral) else tuple(normalized_shape)
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
    """torch.nn.RMSNorm over the last dimension, on rms_norm().  eps is 1e-6 if it
    is not given, where torch's module takes None; None means here what it means
    there, float32's epsilon for rows of any type."""

    def __init__(self, normalized_shape, eps: float | None = 1e-6, elementwise_affine: bool = True, device=None,
                 dtype=None):
        super().__init__(_one_dim(normalized_shape), eps, elementwise_affine, device, dtype)

    def forward(self, x):
        if x.shape[-1:] != self.normalized_shape:
            raise ValueError(f"expected a last dimension of {self.normalized_shape[0]}, got shape {tuple(x.shape)}")
        return rms_norm(x, self.weight, torch.finfo(torch.float32).eps if self.eps is None else self.eps)


class FlashDropout(torch.nn.Module):
    """torch.nn.Dropout on dropout(); `counter` (shared between modules or not)
    gives every call its mask, and a recomputed call the mask of its first run.
    Copies of the module share the counter, so they draw masks of their own.
    What resumes the masks is the counter's state_dict(), saved beside the
    model's, which holds nothing of it."""

    def __init__(self, p: float, counter: DropoutCounter):
        super().__init__()
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"the drop probability must lie in [0, 1], got {p}")
        self.p, self.counter = float(p), counter

    def forward(self, x):
        if not self.training or self.p == 0.0:
            return x
        return dropout(x, self.p, **self.counter.next())

    def __deepcopy__(self, memo):
        memo.setdefault(id(self.counter), self.counter)
        new = memo[id(self)] = self.__class__.__new__(self.__class__)
        new.__dict__.update(copy.deepcopy(self.__dict__, memo))
        return new

    def extra_repr(self) -> str:
        return f"p={self.p}"
