"""Norms of rows whose sums, but not their means, pass float32's range.  The
bounds are those of rows_helpers.py: the errors they count are relative, and no
power of two changes them."""

import numpy as np
import pytest
import torch

from precision_optimizer_state_amd import binding as B
from precision_optimizer_state_amd import nn
from rows_helpers import DTYPES, check_backward, check_forward, host

pytestmark = pytest.mark.gpu

# one lane's reach, a wave's, a workgroup's, an odd length, rows that are read from memory again
COLS = [8, 100, 768, 4096, 8191, 16384, 20000]


def run(kind, cols, dtype, scale, loc=0.0, rows=7):
    rng = np.random.default_rng([cols, int(abs(np.log2(scale)))])
    dt, eps = DTYPES[dtype], 1e-5
    x = torch.from_numpy(((rng.normal(size=(rows, cols)) + loc) * scale).astype(np.float32)).to(dt).cuda()
    w = torch.from_numpy(rng.normal(1, 0.3, cols).astype(np.float32)).to(dt).cuda()
    b = torch.from_numpy(rng.normal(0, 0.3, cols).astype(np.float32)).to(dt).cuda() if kind == "layer" else None
    dy = torch.from_numpy(rng.normal(size=(rows, cols)).astype(np.float32)).to(dt).cuda()
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    mean = torch.empty(rows, device="cuda") if kind == "layer" else None
    B.fo_norm_forward(x, y, kind, w, b, eps, mean_out=mean, rstd_out=rstd)
    leaves = [t.requires_grad_(True) for t in (x, w, b) if t is not None]
    out = nn.layer_norm(x, w, b, eps) if kind == "layer" else nn.rms_norm(x, w, eps)
    assert torch.equal(out, y)
    return x, w, b, dy, y, rstd, torch.autograd.grad(out, leaves, dy)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sums_past_the_range_of_float32(kind, cols, dtype):
    # mean squares up to 4^2 * 1.2e37, within float32; their sums over the row are not.  Normal
    # values of 2^61.5 stay under 2^64, whose square is float32's end
    x, w, b, dy, y, rstd, grads = run(kind, cols, dtype, 2.0 ** 61.5)
    assert (rstd > 0).all()
    check_forward("y", y, host(x), host(w), None if b is None else host(b), 1e-5, kind)
    got = dict(zip(("d", "dweight", "dbias"), grads))
    check_backward("", got, host(dy), host(x), host(w), 1e-5, kind)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_means_of_the_largest_values(cols, dtype):
    # the sum of a row passes 2^128, its mean is 2^125.6 and the spread about it 2^122
    for kind in ("layer", "rms"):
        _, _, b, _, y, rstd, grads = run(kind, cols, dtype, 2.0 ** 122, loc=12.0)
        # squares past float32's range: r = 0, so y is the bias and the rows' gradient 0
        assert (rstd == 0).all()
        assert torch.equal(y, torch.zeros_like(y) if b is None else b.expand_as(y))
        assert (grads[0] == 0).all() and all(torch.isfinite(g).all() for g in grads)


@pytest.mark.parametrize("cols", COLS)
def test_both_sides_of_the_limit(cols):
    # rows of one magnitude a with alternating signs: the mean square is a^2 exactly, and float32's
    # range ends at 2^128
    for a, fits in ((2.0 ** 63.99, True), (2.0 ** 64.01, False)):
        x = torch.full((3, cols), a, device="cuda")
        x[:, 1::2] *= -1
        y = nn.rms_norm(x)
        assert torch.equal(y == 0, torch.full_like(y, not fits, dtype=torch.bool)), (cols, a)
        if fits:
            check_forward("y", y, host(x), None, None, 1e-6, "rms")


def test_infinities_stay_not_finite():
    x = torch.randn(4, 5000, device="cuda") * 2.0 ** 61
    x[1, 7], x[2, 9] = float("inf"), float("nan")
    for y in (nn.rms_norm(x), nn.layer_norm(x)):
        assert torch.isfinite(y[[0, 3]]).all() and torch.isnan(y[1, 7]) and torch.isnan(y[2]).all()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_small_rows_without_eps(cols, kind):
    # squares of values of 2^-50, scaled by a power of two near 1 / cols (2^-16 at most), stay normal
    rng = np.random.default_rng(cols)
    x = torch.from_numpy((rng.normal(size=(5, cols)) * 2.0 ** -50).astype(np.float32)).cuda()
    y = nn.layer_norm(x, eps=0.0) if kind == "layer" else nn.rms_norm(x, eps=0.0)
    check_forward("y", y, host(x), None, None, 0.0, kind)
