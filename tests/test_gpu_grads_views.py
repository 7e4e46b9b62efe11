"""Gradient clipping into tensors that are no stretch of memory of their own: what cannot be
written is refused before anything is."""

import pytest
import torch

from precision_optimizer_state_amd import grads
from step_helpers import generator, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(4, 8), (8,)])
def test_an_output_whose_elements_share_memory_is_refused_first(shape):
    """An expanded tensor: nothing is scaled, whatever stands before it in the list."""
    gen = generator(60)
    for where in (0, 1):
        a = normal(gen, 100)
        shared = torch.ones(1, device="cuda").expand(shape)
        before, version = a.clone(), a._version
        listed = [shared, a] if where == 0 else [a, shared]
        with pytest.raises(RuntimeError, match="single memory location"):
            grads.clip_grads(listed, 0.1)
        assert torch.equal(a, before) and a._version == version
        out = [shared if t is shared else torch.zeros_like(a) for t in listed]
        with pytest.raises(RuntimeError, match="single memory location"):
            grads.clip_grads([torch.ones(shape, device="cuda") if t is shared else a for t in listed], 0.1, out=out)
        assert not any(o.any() for o in out if o is not shared)
    # as an input it is fine
    got, norm = grads.clip_grads([shared], 1.0, out=[torch.empty(shape, device="cuda")])
    assert abs(float(norm) - shared.numel() ** 0.5) < 1e-5 and (got[0] - 1 / norm).abs().max() < 1e-5


def test_slices_made_under_inference_mode():
    """... are scaled where they lie, as whole tensors are."""
    gen = generator(61)
    with torch.inference_mode():
        wide = normal(gen, 40, 30)
        whole = wide.clone()
    part = wide[:, 3:20]
    want = part / part.norm() * 0.5
    rest = wide[:, 20:].clone()
    for t in (part, whole):
        grads.clip_grads([t], 0.5)
    assert (part - want).abs().max() < 1e-6 and torch.equal(wide[:, 20:], rest)
    assert abs(float(grads.grad_norm([part])) - 0.5) < 1e-4 and abs(float(grads.grad_norm([whole])) - 0.5) < 1e-4
