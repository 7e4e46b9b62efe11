"""Pins of the row operators' oracle (CPU): the generator against its published
test vectors, the keep decisions against a scalar transcription and their
rates, the norms against torch in float64, their gradients against autograd and
against differences."""

import numpy as np
import pytest
import torch

from oracle import rows as R


@pytest.mark.parametrize("counter, key, want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((R.M32,) * 4, (R.M32,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, want):
    # the generator's published known-answer vectors (all zeros, all ones, digits of pi)
    assert tuple(R.philox4x32(counter, key)) == want


@pytest.mark.parametrize("rows, cols, first", [(3, 5, 0), (2, 8, 7), (2, 17, (1 << 31) + 3)])
def test_uniforms_element_by_element(rows, cols, first):
    seed, offset = 0x9123456789ABCDEF, 0x1FFFFFFFF
    got = R.uniforms(rows, cols, seed, offset, first)
    per = (cols + 7) // 8
    for r in range(rows):
        for c in range(cols):
            b = (first + r) * per + c // 8
            j = c % 8
            halves = []
            for i in (0, 1):
                w = R.philox4x32((b % 2 ** 32, b // 2 ** 32 + i * 2 ** 31, offset % 2 ** 32, offset // 2 ** 32),
                                 (seed % 2 ** 32, seed // 2 ** 32))[j // 2]
                halves.append(w >> 16 if j % 2 else w & 0xFFFF)
            assert got[r, c] == halves[0] * 65536 + halves[1]


@pytest.mark.parametrize("p", [0.001, 0.1, 0.5, 0.9])
def test_keep_rate(p):
    n = 1 << 20
    kept = R.keep(n // 64, 64, p, 11, 5).mean()
    assert abs(kept - (1 - p)) < 5 * np.sqrt(p * (1 - p) / n)        # five standard deviations


def test_masks_of_other_offsets_seeds_and_rows_differ():
    a = R.keep(64, 64, 0.5, 1, 1)
    for b in (R.keep(64, 64, 0.5, 1, 2), R.keep(64, 64, 0.5, 2, 1), R.keep(64, 64, 0.5, 1, 1, 64)):
        assert abs((a == b).mean() - 0.5) < 0.05


def test_scale_and_threshold():
    assert R.threshold(0.0) == 0 and R.scale(0.0) == 1.0
    assert R.threshold(1.0) == 1 << 32 and R.scale(1.0) == 0.0
    assert R.scale(0.5) == 2.0
    assert abs(R.scale(0.1) * 0.9 - 1) < 2.0 ** -32


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 2), (5, 17)])
def test_norm_against_torch_and_autograd(kind, shape):
    rng = np.random.default_rng(3)
    h, dy, dh = (torch.tensor(rng.normal(size=shape) + 0.5, requires_grad=True) for _ in range(3))
    w, b = (torch.tensor(rng.normal(size=shape[1]), requires_grad=True) for _ in range(2))
    if kind == "layer":
        y = torch.nn.functional.layer_norm(h, shape[1:], w, b, 1e-5)
    else:
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-5) * w
    got, _, _ = R.norm_forward(h.detach(), w.detach(), b.detach() if kind == "layer" else None, 1e-5, kind)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    gh, gw = torch.autograd.grad([y, h], [h, w], [dy.detach(), dh.detach()])
    d, dw, db = R.norm_backward(dy.detach(), h.detach(), w.detach(), 1e-5, kind, dh.detach())
    np.testing.assert_allclose(d, gh.numpy(), rtol=1e-9, atol=1e-9)
    np.testing.assert_allclose(dw, gw.numpy(), rtol=1e-9, atol=1e-9)
    np.testing.assert_allclose(db, dy.detach().sum(0).numpy(), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradient_against_differences(kind):
    rng = np.random.default_rng(4)
    h, w, dy = rng.normal(size=(4, 9)), rng.normal(size=9), rng.normal(size=(4, 9))
    d, dw, _ = R.norm_backward(dy, h, w, 1e-5, kind)
    step = 1e-5

    def loss(hh, ww):
        return (R.norm_forward(hh, ww, None, 1e-5, kind)[0] * dy).sum()

    # central differences: truncation step^2 ~ 1e-10 times third derivatives of a few hundred
    # at most, rounding 2^-53 * 40 / step ~ 1e-9
    for i in np.ndindex(h.shape):
        e = np.zeros_like(h)
        e[i] = step
        assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * step) - d[i]) < 1e-6
    for i in range(9):
        e = np.zeros_like(w)
        e[i] = step
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * step) - dw[i]) < 1e-6
