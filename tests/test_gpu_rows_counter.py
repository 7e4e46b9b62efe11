"""FlashDropout and the counter's keys in recomputed forward passes on the GPU,
against the same model without recomputation."""

import copy

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from precision_optimizer_state_amd import nn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("reentrant", [True, False])
def test_modules_in_recomputed_segments(reentrant):
    def model():
        torch.manual_seed(1)
        counter = nn.DropoutCounter(seed=6)

        def segment():
            return torch.nn.Sequential(nn.FlashDropout(0.3, counter), nn.FlashLayerNorm(72, device="cuda"),
                                       torch.nn.Linear(72, 72, device="cuda"), nn.FlashDropout(0.5, counter))
        return counter, torch.nn.ModuleList(segment() for _ in range(3))

    out = []
    for recompute in (False, True):
        counter, segments = model()
        x = torch.randn(50, 72, device="cuda", generator=torch.Generator("cuda").manual_seed(5)).requires_grad_(True)
        for _ in range(2):                               # two steps
            y = x
            for s in segments:
                y = checkpoint(s, y, use_reentrant=reentrant) if recompute else s(y)
            y.square().sum().backward()
        assert counter.offset == 12
        out.append([y, x.grad] + [q.grad for q in segments.parameters()])
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("reentrant", [True, False])
def test_joins_with_keys_taken_inside(reentrant):
    counter = nn.DropoutCounter(seed=6)
    w = torch.randn(40, device="cuda", requires_grad=True)

    def block(h, y):
        return nn.dropout_add_rms_norm(y * 2, h, w, p=0.4, **counter.next())

    out = []
    for recompute in (False, True):
        counter.offset, w.grad = 0, None
        x = torch.arange(800.0, device="cuda").view(20, 40).sin().requires_grad_(True)
        h, y = x, x
        for _ in range(3):
            h, y = checkpoint(block, h, y, use_reentrant=reentrant) if recompute else block(h, y)
        (h * y).sum().backward()
        out.append((h, y, x.grad, w.grad))
    assert counter.offset == 3 and all(torch.equal(a, b) for a, b in zip(*out))


def test_copies_of_a_module_draw_masks_of_their_own():
    block = torch.nn.Sequential(nn.FlashDropout(0.5, nn.DropoutCounter(seed=2)))
    x = torch.ones(64, 64, device="cuda")
    masks = [copy.deepcopy(block)(x) for _ in range(3)] + [block(x)]
    for i, a in enumerate(masks):
        assert torch.equal(a, nn.dropout(x, 0.5, 2, i))
