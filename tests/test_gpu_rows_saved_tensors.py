"""What the row operators keep for their backward passes, through hooks on saved tensors:
the same gradients where the values come back, and a refusal where something else does."""

import pytest
import torch

from precision_optimizer_state_amd import nn
from test_gpu_saved_tensors import CHANGES, gradients, strided

pytestmark = pytest.mark.gpu


def inputs(dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(80)
    x, r = (torch.randn(40, 72, generator=gen, device="cuda").to(dtype).requires_grad_(True) for _ in range(2))
    w, b = (torch.randn(72, generator=gen, device="cuda").to(dtype).requires_grad_(True) for _ in range(2))
    return x, r, w, b


def state():
    return torch.tensor([3, 1 << 32], device="cuda")


# operator -> how many tensors it keeps
OPS = {
    "layer": (lambda x, r, w, b: nn.layer_norm(x, w, b) + 0 * r, 3),
    "rms": (lambda x, r, w, b: nn.rms_norm(x, w) + 0 * r + 0 * b, 3),
    "join": (lambda x, r, w, b: torch.cat(nn.dropout_add_layer_norm(x, r, w, b, p=0.3, seed=5, state=state())), 4),
    "dropout": (lambda x, r, w, b: nn.dropout(x, 0.3, 5, 1, state()) + 0 * r + 0 * w + 0 * b, 1),
}


@pytest.mark.parametrize("op", list(OPS))
def test_the_same_values_elsewhere(op):
    args = inputs()
    want = gradients(OPS[op][0], args)
    for pack, unpack in ((lambda t: t.cpu(), lambda t: t.cuda()),
                         (lambda t: t.clone(), lambda t: t if t.dtype == torch.int64 else strided(t))):
        for a, b in zip(gradients(OPS[op][0], args, pack, unpack), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("change", list(CHANGES))
@pytest.mark.parametrize("op", list(OPS))
def test_something_else_is_refused(op, change):
    args, (call, tensors) = inputs(), OPS[op]
    refused = 0
    for k in range(tensors):
        n = []

        def pack(t):
            n.append(0)
            return len(n) - 1, t

        def unpack(kept):
            return CHANGES[change](kept[1]) if kept[0] == k else kept[1]

        try:
            gradients(call, args, pack, unpack)
        except (ValueError, RuntimeError) as e:
            assert any(s in str(e) for s in ("GPU", "came back", "agree", "shape", "not supported", "2 int64", "a gradient is")), e
            refused += 1
        else:
            # a weight of another type is one that the kernels take; its gradient comes in the leaf's
            assert change == "of another type" and op == "rms"
    assert refused >= tensors - 1
    torch.cuda.synchronize()
