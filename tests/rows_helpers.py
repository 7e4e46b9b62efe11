"""Inputs and error bounds of the row operators' GPU tests.

Every bound is an a-priori one.  With U = 2^-24 (half a float32 step) and E_T
half a step of the output's type relative to the value (bfloat16 2^-8 ... as
torch.finfo(T).eps / 2), an output of T may be off by E_T |want| (plus half the
type's smallest subnormal) for its one rounding, plus the float32 error of what
was rounded.  A float32 sum of n terms in any order of depth D is off by at
most D U sum|terms| (first order).  A row's sums have depth at most
cols / 256 + 32 here (terms added one after another by one lane, then a tree of
at most 10 levels and at most 16 wave sums), sums over rows rows / 256 + 96.

First-order propagation, with u = (h - m) r and H = mean|h| * r:
  m is off by D U mean|h|, r by a relative (D / 2 + 4) U plus the same error of
  m at second order, so u is off by at most (D + 8) U (|u| + H);
  y = u w + b: that times |w|, and 2 U (|u w| + |b|) for its own operations;
  d: the three terms of r (g - mean g - u mean(g u)), each with D + 12 roundings
  and the error of u in both its places, and one more for adding dh;
  dw = sum dy u: depth of the sum plus the error of u.
"""

from __future__ import annotations

import numpy as np
import torch

from oracle import rows as R

U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


def half_step(dtype, want):
    info = torch.finfo(dtype)
    tiny = info.tiny * info.eps / 2                     # half the smallest subnormal
    # past the midpoint above the largest finite value a rounding gives infinity
    return info.eps / 2 * np.abs(want) + tiny


def host(t):
    return t.detach().to(torch.float64).cpu().numpy()


def check(name, got, want, dtype, f32_error):
    got = host(got) if torch.is_tensor(got) else got
    bound = half_step(dtype, want) * (1 + 2.0 ** -8) + f32_error
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} outside their bound; first at {i}: got {got[i]!r}, "
                             f"want {want[i]!r}, bound {np.broadcast_to(bound, want.shape)[i]!r}")


def row_depth(cols):
    return cols / 256 + 32


def col_depth(rows):
    return rows / 256 + 96


def check_forward(name, y, h, weight, bias, eps, kind):
    """y against the norm of h (host float64 rows, as stored)."""
    want, mean, rstd = R.norm_forward(h, weight, bias, eps, kind)
    w = np.ones(h.shape[1]) if weight is None else np.abs(weight)
    b = np.zeros(h.shape[1]) if bias is None else np.abs(bias)
    u, big = np.abs(h - mean) * rstd, np.abs(h).mean(1, keepdims=True) * rstd
    err = U * ((row_depth(h.shape[1]) + 8) * (u + big) * w + 2 * (u * w + b))
    check(name, y, want, y.dtype, err)


def check_backward(name, grads, dy, h, weight, eps, kind, dh=None, drop=None):
    """grads: dict with some of d, dx, dweight, dbias; drop: (p, seed, offset)."""
    d, dw, db = R.norm_backward(dy, h, weight, eps, kind, dh)
    _, mean, rstd = R.norm_forward(h, None, None, eps, kind)
    depth = row_depth(h.shape[1])
    g = np.abs(dy) if weight is None else np.abs(dy * weight)
    ub = np.abs(h - mean) * rstd + np.abs(h).mean(1, keepdims=True) * rstd          # |u| + H
    err = 2 * U * (depth + 12) * rstd * (g + g.mean(1, keepdims=True) + ub * (g * ub).mean(1, keepdims=True))
    if dh is not None:
        err = err + 2 * U * (np.abs(dh) + np.abs(d))
    if grads.get("d") is not None:
        check(name + " d", grads["d"], d, grads["d"].dtype, err)
    if grads.get("dx") is not None:
        p, seed, offset = drop
        k = R.keep(*h.shape, p, seed, offset)
        want, err = np.where(k, d * R.scale(p), 0.0), np.where(k, (err + 2 * U * np.abs(d)) * R.scale(p), 0.0)
        check(name + " dx", grads["dx"], want, grads["dx"].dtype, err)
    rd = col_depth(h.shape[0])
    if grads.get("dweight") is not None:
        err = U * (rd + depth + 8) * (np.abs(dy) * ub).sum(0)
        check(name + " dweight", grads["dweight"], dw, grads["dweight"].dtype, err)
    if grads.get("dbias") is not None:
        check(name + " dbias", grads["dbias"], db, grads["dbias"].dtype, U * rd * np.abs(dy).sum(0))


def matrix(rng, rows, cols, dtype, loc=0.0, spread=1.0, pad=0, lead=0):
    """rows x cols of dtype on the GPU; with pad/lead a slice of a wider matrix."""
    a = torch.from_numpy(rng.normal(loc, spread, size=(rows, cols + pad + lead)).astype(np.float32))
    return a.to(dtype).cuda()[:, lead:lead + cols]
