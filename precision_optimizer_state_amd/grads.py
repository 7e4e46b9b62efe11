"""The norm of a model's gradients taken together, and clipping by it.

Clipping stands between the backward pass and the optimizers of this package:

    loss.backward()
    norm = clip_grad_norm_(model.parameters(), 1.0)     # or opt.clip_grad_norm_(1.0)
    opt.step()

or, where gradients are summed in single precision over several micro-batches,
from those sums into the 16-bit gradients that the optimizers read:

    clip_grads(sums, 1.0, out=[p.grad for p in params])

All arithmetic runs in the HIP library (fo_grad_norm and fo_grad_clip in
include/foamd.h); a host extension (csrc/fo_step_torch.cpp) marshals the
tensors.  Norms are summed in float64, so they neither overflow nor lose small
gradients among large ones, and repeat bit for bit.  Calls go to torch's current
stream and never synchronise (but for error_if_nonfinite), so they can be
captured into HIP graphs.
"""

from __future__ import annotations

import math

import torch

from . import binding as B
from .nn import _step_ext

_ORDERS = {2.0: B.FO_NORM_2, 1.0: B.FO_NORM_1, math.inf: B.FO_NORM_MAX}


def _order(norm_type) -> int:
    order = _ORDERS.get(float(norm_type))
    if order is None:
        raise ValueError(f"norm_type must be 2, 1 or inf, got {norm_type}")
    return order


def _bound(max_norm) -> float:
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"max_norm must be >= 0, got {max_norm}")
    return max_norm


def _listed(tensors) -> list:
    return [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)


def grad_norm(grads, norm_type: float = 2.0) -> torch.Tensor:
    """The norm of all elements of `grads` (a tensor or an iterable of them, of
    bfloat16, float16 or float32, mixed or not) as one vector: a float32 scalar
    on the GPU.  norm_type: 2, 1 or inf.  An empty list has norm 0.  The norm has no
    derivatives: a backward pass through it is refused."""
    return _step_ext().grad_norm(_listed(grads), _order(norm_type))


def clip_grads(grads, max_norm: float, norm_type: float = 2.0, *, out=None, error_if_nonfinite: bool = False):
    """Scale gradients by min(1, max_norm / (norm + 1e-6)): (clipped, norm).

    `out`: tensors of the gradients' shapes to write, of the same or other
    types (each element is rounded once); without it the gradients themselves
    are scaled.  No tensor may be listed twice.  A NaN norm makes every gradient
    NaN, an infinite one makes them 0 (and the infinite elements NaN), as torch's
    clipping does; max_norm = inf leaves them as they are.  error_if_nonfinite waits
    for the norm and raises, with nothing written, if it is not finite."""
    grads = _listed(grads)
    outs = grads if out is None else _listed(out)
    max_norm, order = _bound(max_norm), _order(norm_type)
    if error_if_nonfinite:
        norm = _step_ext().grad_norm(grads, order).item()
        if not math.isfinite(norm):
            raise RuntimeError(f"the norm of the gradients is {norm}, so they cannot be clipped")
    return outs, _step_ext().clip(grads, outs, max_norm, order)


def clip_grad_norm_(parameters, max_norm: float, norm_type: float = 2.0,
                    error_if_nonfinite: bool = False) -> torch.Tensor:
    """torch.nn.utils.clip_grad_norm_ on clip_grads(): scale the .grad of
    `parameters` in place; returns the norm before clipping.  Where the bound holds
    gradients keep their bits, and are not written unless they are slices that are not
    one stretch of memory: those are clipped as copies and written back."""
    grads = [p.grad for p in _listed(parameters) if p.grad is not None]
    return clip_grads(grads, max_norm, norm_type, error_if_nonfinite=error_if_nonfinite)[1]
