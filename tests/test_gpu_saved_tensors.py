"""What the loss and the gated block keep for their backward passes, through hooks on saved
tensors: the same gradients where the values come back, in whatever layout, and a refusal
where something else does."""

import pytest
import torch

from precision_optimizer_state_amd import nn
from step_helpers import TYPES, generator, normal

pytestmark = pytest.mark.gpu


def loss_none(x, w, t):
    return nn.linear_cross_entropy(x, w, t, reduction="none")


def loss_mean(x, w, t):
    return nn.linear_cross_entropy(x, w, t)


def gated(x, a, b):
    return nn.gated_linear(x, a, b)


def inputs(op, dtype="bf16"):
    gen = generator(70)
    x = normal(gen, 40, 72, dtype=TYPES[dtype])
    w = normal(gen, 90, 72, scale=0.1, dtype=TYPES[dtype])
    last = normal(gen, 90, 72, scale=0.1, dtype=TYPES[dtype]) if op is gated else torch.randint(90, (40,), generator=gen, device="cuda")
    return [t.requires_grad_(t.is_floating_point()) for t in (x, w, last)]


def gradients(op, args, pack=None, unpack=None):
    if pack:
        with torch.autograd.graph.saved_tensors_hooks(pack, unpack):
            y = op(*args)
    else:
        y = op(*args)
    return torch.autograd.grad(y.float().sum(), [a for a in args if a.requires_grad])


def strided(t):
    """The same values, apart from each other."""
    wide = torch.zeros(t.shape + (3,), dtype=t.dtype, device=t.device)
    wide[..., 1] = t
    return wide[..., 1]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("op", [loss_none, loss_mean, gated])
def test_the_same_values_elsewhere(op, dtype):
    args = inputs(op, dtype)
    want = gradients(op, args)
    for pack, unpack in ((lambda t: t.cpu(), lambda t: t.cuda()), (lambda t: t.clone(), strided)):
        for a, b in zip(gradients(op, args, pack, unpack), want):
            assert torch.equal(a, b)


CHANGES = {
    "on the host": lambda t: t.cpu(),
    "of another type": lambda t: t.int() if t.dtype == torch.int64 else t.half() if t.dtype != torch.float16 else t.float(),
    "shorter": lambda t: t.flatten()[:-1] if t.numel() > 1 else t.repeat(2),
    "fewer rows": lambda t: t[:-1] if t.dim() and t.shape[0] > 1 else t.reshape(1, 1),
}


@pytest.mark.parametrize("change", list(CHANGES))
@pytest.mark.parametrize("op, tensors", [(loss_none, 4), (loss_mean, 5), (gated, 5)])
def test_something_else_is_refused(op, tensors, change):
    args = inputs(op)
    seen = []
    gradients(op, args, lambda t: seen.append(t) or t, lambda t: t)
    # (the first saved tensors are the operator's; .float() and .sum() keep none)
    assert len(seen) == tensors
    for k in range(tensors):
        n = []

        def pack(t):
            n.append(0)
            return len(n) - 1, t

        def unpack(kept):
            return CHANGES[change](kept[1]) if kept[0] == k else kept[1]

        with pytest.raises((ValueError, RuntimeError), match="GPU|came back|agree|int64|shape|not supported"):
            gradients(op, args, pack, unpack)
    torch.cuda.synchronize()
