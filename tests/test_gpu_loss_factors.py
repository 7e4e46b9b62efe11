"""nn.linear_cross_entropy where the gradient of one token's loss is infinite or NaN: what
the other tokens' gradients may not see of it."""

import pytest
import torch

from step_helpers import TYPES, Loss, check, generator
from test_gpu_loss import make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", [1024.0, 1.0, 1e-3])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_one_token_without_a_finite_factor(bad, size, dtype):
    """The other tokens' gradients are those of a factor of 0 in its place, to the bit, and
    within their bounds: in half precision they neither overflow nor lose their digits."""
    x, w, t = make(30, 40, 96, 150, dtype)
    gen = generator(31)
    dloss = size * (0.5 + torch.rand(40, generator=gen, device="cuda"))
    dloss[9] *= -1
    dloss[4] = 0.0
    _, dx0, dw0, _ = run(x, w, t, "none", dloss=dloss)
    ref = Loss(x, w, t, "none", 0.0, -100, dloss)
    check("dx", dx0, ref.dx, ref.d_dx)
    check("dw", dw0, ref.dw, ref.d_dw)
    dloss[4] = bad
    _, dx, dw, _ = run(x, w, t, "none", dloss=dloss)
    keep = torch.arange(40, device="cuda") != 4
    assert torch.equal(dx[keep], dx0[keep])
    assert not torch.isfinite(dx[4]).any() and not torch.isfinite(dw).any()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_an_infinite_factor_alone(dtype):
    """The other factors are 0: so are their gradients."""
    x, w, t = make(32, 20, 64, 70, dtype)
    dloss = torch.zeros(20, device="cuda")
    dloss[3] = float("inf")
    _, dx, _, _ = run(x, w, t, "none", dloss=dloss)
    keep = torch.arange(20, device="cuda") != 3
    assert not dx[keep].any() and not torch.isfinite(dx[3]).any()
