"""Construction of the norm modules, without a GPU."""

import numpy as np
import pytest
import torch

from precision_optimizer_state_amd import nn


def test_eps_of_an_rms_norm(monkeypatch):
    seen = []
    monkeypatch.setattr(nn, "rms_norm", lambda x, weight=None, eps=1e-6: seen.append(eps) or x)
    x = torch.ones(2, 8)
    for args, want in (({}, 1e-6), ({"eps": 1e-3}, 1e-3), ({"eps": None}, torch.finfo(torch.float32).eps)):
        for dtype in (torch.float32, torch.bfloat16):
            module = nn.FlashRMSNorm(8, dtype=dtype, **args)
            module(x.to(dtype))
            assert seen.pop() == want and module.eps == args.get("eps", 1e-6)
            repr(module)


@pytest.mark.parametrize("cls", [nn.FlashLayerNorm, nn.FlashRMSNorm])
@pytest.mark.parametrize("size", [8, (8,), [8], torch.Size([8]), np.int64(8)])
def test_sizes_as_torch_takes_them(cls, size):
    assert cls(size).normalized_shape == (8,)
