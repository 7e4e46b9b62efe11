"""References in 64 bits and error bounds of the tests of clipping, linear cross entropy
and the gated block.

Every bound is an a-priori one.  U = 2^-24 is half a float32 step relative to the value,
E_T = torch.finfo(T).eps / 2 that of the outputs' type.

A product's sum of K float32 terms, added in any order by matrix instructions whose inner
additions may truncate (2 U each), is off by at most 2 (K + 2) U sum |terms|: S below.

linear cross entropy, with dz = the bound of a logit, A = its largest value in the row:
  exponentials: the argument z log2(e) - n carries the constant's and the fused
    operation's rounding, U |z log2 e| each, the hardware's exponential 2 U: relative
    e = 2 U (1.45 A + 4);
  their sum over V places has a chain of at most V / 4096 + 200 additions;
  lse: dz + e + that chain's U + 4 U (|lse| + 1) for logarithm and joining;
  a row's loss: lse + (1 - s) dz + s (dz + (V / 4096 + 200) U mean |z|) + 4 U (|lse| + |z_t| + mean |z|).
  P = (softmax - y) unit: relative to softmax dz + the error of lse + e, plus 4 U of
    (softmax + y + s / V), plus its rounding to T: E_T |P| and, in half precision, which
    holds it times 2^15, 2^-25 2^-15 below its normal numbers;
  dx, dW: |P|'s error through the product, S of the product, E_T of the result.

the gated block, with S of both products: act(g) has a slope of at most 1.13 in absolute
value and its own evaluation's error 16 U |g|; act' has one of at most 1 and 32 U (1 + |g|).
"""

from __future__ import annotations

import math

import torch

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


def half_step(dtype, want):
    info = torch.finfo(dtype)
    return info.eps / 2 * want.abs() + info.tiny * info.eps / 2


def check(name, got, want, bound):
    got, want = got.detach().double(), want.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = (got - want).abs()
    ok = (off <= bound) | (got.isnan() & want.isnan())
    if not bool(ok.all()):
        i = tuple(int(v) for v in torch.nonzero(~ok)[0]) if got.dim() else ()
        bound = torch.as_tensor(bound, device=got.device, dtype=torch.float64).expand_as(want)
        raise AssertionError(f"{name}: {int((~ok).sum())} of {got.numel()} outside their bound; first at {i}: got "
                             f"{got[i].item()!r}, want {want[i].item()!r}, bound {bound[i].item()!r}")


def product_bound(a, b):
    """S of a b^T."""
    return 2 * (a.shape[1] + 2) * U * (a.abs() @ b.abs().t())


class Loss:
    """The reference of one call: loss, dx, dw in float64, and their bounds."""

    def __init__(self, x, w, target, reduction="mean", smoothing=0.0, ignore=-100, dloss=None):
        self.dtype = x.dtype
        x, w = x.detach().double().reshape(-1, x.shape[-1]), w.detach().double()
        t = target.reshape(-1)
        n, V = x.shape[0], w.shape[0]
        counted = t != ignore
        idx = torch.where(counted, t, torch.zeros_like(t))
        x = torch.where(counted[:, None], x, 0.0)             # what others hold has no part in anything
        z = x @ w.t()
        dz = product_bound(x, w)
        dmax = dz.max(1).values
        A = z.abs().max(1).values
        lse = torch.logsumexp(z, 1)
        e = 2 * U * (1.45 * A + 4)
        chain = (V / 4096 + 200) * U
        d_lse = dmax + e + chain + 4 * U * (lse.abs() + 1)
        zt, mean, mean_abs = z.gather(1, idx[:, None])[:, 0], z.mean(1), z.abs().mean(1)
        rows = lse - (1 - smoothing) * zt - smoothing * mean
        d_rows = d_lse + dmax + smoothing * chain * mean_abs + 4 * U * (lse.abs() + zt.abs() + mean_abs)
        rows, d_rows = torch.where(counted, rows, 0.0), torch.where(counted, d_rows, 0.0)
        count = counted.sum()
        if reduction == "none":
            self.loss, self.d_loss = rows.view(target.shape), d_rows.view(target.shape)
        else:
            div = count.double() if reduction == "mean" else 1.0
            self.loss = rows.sum() / div
            self.d_loss = d_rows.sum() / div + 2 * U * self.loss.abs()
        if dloss is None:
            return
        f = dloss.double().reshape(-1).expand(n) / (count if reduction == "mean" else 1)
        f = torch.where(counted, f, 0.0)
        top = f.abs().max().clamp(min=1e-300)
        unit = (f / top)[:, None]
        p = torch.softmax(z, 1)
        y = torch.zeros_like(p).scatter_(1, idx[:, None], 1 - smoothing) + smoothing / V
        P = (p - y) * unit
        d_p = (p * (dz + d_lse[:, None] + e[:, None]) + 4 * U * (p + y)) * unit.abs()
        if self.dtype != torch.float32:
            d_p = d_p * (1 + 2.0 ** -8) + torch.finfo(self.dtype).eps / 2 * P.abs()
        if self.dtype == torch.float16:
            d_p = d_p + 2.0 ** -40
        d_p = torch.where(counted[:, None], d_p, 0.0)
        self.dx, self.dw = P @ w * top, P.t() @ x * top
        half = torch.finfo(self.dtype).eps / 2
        for name, got, a, da, b in (("dx", self.dx, P, d_p, w), ("dw", self.dw, P.t(), d_p.t(), x)):
            inner = (da @ b.abs() + 2 * (a.shape[1] + 40) * U * (a.abs() @ b.abs())) * top * (1 + half + 4 * U)
            inner = inner + 8 * U * got.abs()                 # the factors' own roundings
            setattr(self, "d_" + name, inner + half_step(self.dtype, got) * (1 + 2.0 ** -7))


def activation(name, g):
    """(act, act') in float64"""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-g * math.sqrt(0.5))
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


class Gated:
    def __init__(self, x, gate, up, act="silu", dy=None):
        self.dtype = x.dtype
        shape = x.shape
        x, gate, up = (a.detach().double() for a in (x.reshape(-1, x.shape[-1]), gate, up))
        g, u = x @ gate.t(), x @ up.t()
        dg_, du_ = product_bound(x, gate), product_bound(x, up)
        a, slope = activation(act, g)
        d_a = 1.13 * dg_ + 16 * U * g.abs()
        y = a * u
        half = torch.finfo(self.dtype).eps / 2
        d_y = d_a * (u.abs() + du_) + a.abs() * du_ + 2 * U * y.abs()
        self.y = y.view(*shape[:-1], -1)
        self.d_y = (d_y * (1 + half) + half_step(self.dtype, y) * (1 + 2.0 ** -7)).view(self.y.shape)
        if dy is None:
            return
        dy = dy.double().reshape(-1, gate.shape[0])
        dg, du = dy * u * slope, dy * a
        e_dg = dy.abs() * (du_ * slope.abs() + (u.abs() + du_) * (dg_ + 32 * U * (1 + g.abs()))) + 4 * U * dg.abs()
        e_du = dy.abs() * d_a + 2 * U * du.abs()
        if self.dtype != torch.float32:
            e_dg = e_dg * (1 + half) + half_step(self.dtype, dg)
            e_du = e_du * (1 + half) + half_step(self.dtype, du)

        def product(terms):
            want = sum(p @ q for p, _, q in terms)
            K = sum(p.shape[1] for p, _, _ in terms)
            err = sum(e @ q.abs() for _, e, q in terms) + 2 * (K + 40) * U * sum(p.abs() @ q.abs() for p, _, q in terms)
            return want, err * (1 + half) + half_step(self.dtype, want) * (1 + 2.0 ** -7)

        self.dx, self.d_dx = product([(dg, e_dg, gate), (du, e_du, up)])
        self.dx, self.d_dx = self.dx.view(shape), self.d_dx.view(shape)
        self.dgate, self.d_dgate = product([(dg.t(), e_dg.t(), x)])
        self.dup, self.d_dup = product([(du.t(), e_du.t(), x)])


def normal(gen, *shape, scale=1.0, dtype=torch.float32, pad=0, lead=0):
    """On the GPU; with pad / lead rows are slices of a wider buffer."""
    wide = shape[:-1] + (shape[-1] + pad + lead,)
    t = (scale * torch.randn(*wide, generator=gen, device="cuda")).to(dtype)
    return t[..., lead:lead + shape[-1]] if pad or lead else t


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)
