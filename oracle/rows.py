"""Oracle of the row operators: dropout's keep decisions, layer norm, RMS norm
and the fused dropout + residual sum + norm, forward and backward, in NumPy
float64 from the formulas.  TEST INFRASTRUCTURE ONLY, as the rest of oracle/.

Keep decisions (element (r, c) of an R x C matrix): chunk b = r * ceil(C / 8)
+ c // 8; W(b, i) = Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random
numbers: as easy as 1, 2, 3", SC 2011) of counter (b mod 2^32, b div 2^32 +
i 2^31, offset mod 2^32, offset div 2^32) under key (seed mod 2^32, seed div
2^32); u = 2^16 * half(W(b, 0), c mod 8) + half(W(b, 1), c mod 8), halves
counted from the low half of word 0; kept where u >= round(2^32 p).
"""

from __future__ import annotations

import numpy as np

M32 = 0xFFFFFFFF


def philox4x32(counter, key, rounds: int = 10):
    """Philox4x32 on Python integers: counter 4 words, key 2 words -> 4 words."""
    c, k = [int(v) for v in counter], [int(v) for v in key]
    for _ in range(rounds):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & M32, (p0 >> 32) ^ c[3] ^ k[1], p0 & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def _philox_array(c0, c1, c2, c3, k0, k1):
    """The same on uint64 arrays of counter words c0, c1: (4, n) words."""
    c = [c0.astype(np.uint64), c1.astype(np.uint64), np.full(c0.shape, c2, np.uint64), np.full(c0.shape, c3, np.uint64)]
    s, m = np.uint64(32), np.uint64(M32)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> s) ^ c[1] ^ np.uint64(k0), p1 & m, (p0 >> s) ^ c[3] ^ np.uint64(k1), p0 & m]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return np.stack(c)


def uniforms(rows: int, cols: int, seed: int, offset: int, first_row: int = 0) -> np.ndarray:
    """u of every element of rows [first_row, first_row + rows), int64 (rows, cols)."""
    per = -(-cols // 8)
    b = np.arange(first_row * per, (first_row + rows) * per, dtype=np.uint64)
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    halves = []
    for i in (0, 1):
        w = _philox_array(b & np.uint64(M32), (b >> np.uint64(32)) + np.uint64(i << 31), offset & M32, offset >> 32,
                          seed & M32, seed >> 32).T                                 # (blocks, 4)
        h = np.stack((w & np.uint64(0xFFFF), w >> np.uint64(16)), axis=2).reshape(rows, per * 8)
        halves.append(h[:, :cols].astype(np.int64))
    return (halves[0] << 16) + halves[1]


def threshold(p: float) -> int:
    return int(np.rint(p * 2.0 ** 32))


def keep(rows, cols, p, seed, offset, first_row=0):
    return uniforms(rows, cols, seed, offset, first_row) >= threshold(p)


def scale(p: float) -> float:
    t = threshold(p)
    return 0.0 if t >= 2 ** 32 else 1.0 / (1.0 - t / 2.0 ** 32)


def dropout(x, p, seed, offset):
    x = np.asarray(x, np.float64)
    return np.where(keep(*x.shape, p, seed, offset), x * scale(p), 0.0)


def norm_forward(h, weight=None, bias=None, eps=1e-5, kind="layer"):
    """(y, mean, rstd) of rows h; mean is 0 for kind "rms"."""
    h = np.asarray(h, np.float64)
    mean = h.mean(1, keepdims=True) if kind == "layer" else np.zeros((h.shape[0], 1))
    rstd = 1.0 / np.sqrt(((h - mean) ** 2).mean(1, keepdims=True) + eps)
    y = (h - mean) * rstd
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def norm_backward(dy, h, weight=None, eps=1e-5, kind="layer", dh=None):
    """(d, dweight, dbias): gradients of h, weight and bias."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    _, mean, rstd = norm_forward(h, eps=eps, kind=kind)
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    u = (h - mean) * rstd
    d = g - u * (g * u).mean(1, keepdims=True)
    if kind == "layer":
        d = d - g.mean(1, keepdims=True)
    d = d * rstd
    if dh is not None:
        d = d + np.asarray(dh, np.float64)
    return d, (dy * u).sum(0), dy.sum(0)
