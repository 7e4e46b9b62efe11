"""Float32 weight gradients of many tokens: sums kept in two levels, whatever the tile.

U = 2^-24.  A sum of n equal terms in one chain is off by up to n U of itself, as roundings
of one binade all go the same way; in two levels, of 512 terms and of the n / 512 sums that
these give, by at most (512 + n / 512) 2 U (the matrix instructions' inner additions may
truncate)."""

import torch
import pytest

from precision_optimizer_state_amd import nn
from step_helpers import U, check, generator

pytestmark = pytest.mark.gpu

N = 32768


def bound(want, terms):
    """... with `terms` U for what the terms themselves are off by"""
    return ((512 + N / 512) * 2 + terms + 4) * U * want.abs()


def test_weight_gradients_of_the_loss():
    """All tokens alike: their gradients of logits are equal, those of places that are no
    target all positive.  A logit is one product, so a probability is off by at most 2 U (1.45 D
    + 4) twice and by the sum's 260 U."""
    gen = generator(50)
    cols = vocab = 4096
    row = 1 + torch.rand(cols, generator=gen, device="cuda")
    w = torch.zeros(vocab, cols, device="cuda")
    w[torch.arange(vocab), torch.arange(cols)] = torch.rand(vocab, generator=gen, device="cuda")
    w.requires_grad_(True)
    t = torch.zeros(N, dtype=torch.int64, device="cuda")
    loss = nn.linear_cross_entropy(row.expand(N, cols), w, t, reduction="sum")
    dw, = torch.autograd.grad(loss, w)
    p = torch.softmax(w.detach().double().diagonal() * row.double(), 0)
    for first in range(1, vocab, 512):
        want = N * p[first:first + 512, None] * row.double()
        check("dw", dw[first:first + 512], want, bound(want, 300))


def test_weight_gradients_of_the_gated_block():
    """All tokens alike, products of one term each: dg = dy u silu'(g), du = dy silu(g), off by
    48 U (1 + g) and 24 U of their values' scale."""
    gen = generator(51)
    cols, features = 4096, 2048
    row = 1 + torch.rand(cols, generator=gen, device="cuda")
    at = torch.arange(features)
    ws = [torch.zeros(features, cols, device="cuda") for _ in range(2)]
    for w in ws:
        w[at, at] = 0.5 + torch.rand(features, generator=gen, device="cuda")
        w.requires_grad_(True)
    y = nn.gated_linear(row.expand(N, cols), *ws)
    got = torch.autograd.grad(y.sum(), ws)
    g, u = (w.detach().double()[at, at] * row.double()[:features] for w in ws)
    s = torch.sigmoid(g)
    for grad, d in zip(got, (u * s * (1 + g * (1 - s)), g * s)):
        want = N * d[:, None] * row.double()
        # silu is at least 0.3 and its slope at least 0.7 here, g at most 3
        check("weight gradient", grad, want, bound(want, 48 * 4 / 0.3))
