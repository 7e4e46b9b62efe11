"""Views that torch negates lazily, as inputs of the row operators."""

import pytest
import torch

from precision_optimizer_state_amd import binding as B
from precision_optimizer_state_amd import nn

pytestmark = pytest.mark.gpu


def negated(t):
    """A view whose value is t and whose memory holds -t."""
    view = torch._neg_view(-t)
    assert view.is_neg() and torch.equal(view, t)
    return view


def test_negated_views_keep_their_sign():
    x, r, dy = (torch.randn(6, 40, device="cuda") for _ in range(3))
    w, b = torch.randn(40, device="cuda"), torch.randn(40, device="cuda")
    for f in (lambda x, r, w, b: nn.dropout(x, 0.3, 1), lambda x, r, w, b: nn.layer_norm(x, w, b),
              lambda x, r, w, b: nn.layer_norm(x[:, 3:30], w[3:30], b[3:30]), lambda x, r, w, b: nn.rms_norm(x, w),
              lambda x, r, w, b: torch.cat(nn.dropout_add_layer_norm(x, r, w, b, p=0.2, seed=3))):
        want = f(x, r, w, b)
        assert torch.equal(f(*map(negated, (x, r, w, b))), want)
        leaves = [t.clone().requires_grad_(True) for t in (x, r, w, b)]
        y = f(*leaves)
        g = torch.randn_like(y)
        plain = torch.autograd.grad(y, leaves, g, allow_unused=True)
        minus = [t.clone().neg_().requires_grad_(True) for t in (x, r, w, b)]
        y = f(*(torch._neg_view(t) for t in minus))
        lazy = torch.autograd.grad(y, minus, negated(g), allow_unused=True)
        assert all((p is None and q is None) or torch.equal(p, -q) for p, q in zip(plain, lazy))
    # the imaginary part of a conjugate, one column wide
    z = torch.randn(8, dtype=torch.complex64, device="cuda").conj()
    part = z.imag.unsqueeze(-1)
    assert part.is_neg() and torch.equal(nn.dropout(part, 0.5, 4), nn.dropout(part.clone(), 0.5, 4))


def test_negated_states_and_raw_arguments_are_refused():
    x = torch.randn(6, 40, device="cuda")
    state = torch.tensor([1, 2], device="cuda")
    with pytest.raises(ValueError, match="negated"):
        nn.dropout(x, 0.5, 1, state=torch._neg_view(state))
    y = torch.empty_like(x)
    for args in ((torch._neg_view(x), y), (torch._neg_view(x)[:, 1:], y[:, 1:].clone()), (x, torch._neg_view(y))):
        with pytest.raises(ValueError, match="negated"):
            B.fo_dropout(*args, B.dropout_key(0.5, 1))
    with pytest.raises(ValueError, match="negated"):
        B.fo_norm_forward(x, y, weight=torch._neg_view(x[0]))
