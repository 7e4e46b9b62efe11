"""The norm modules next to torch's on the GPU."""

import pytest
import torch

from precision_optimizer_state_amd import nn
from rows_helpers import DTYPES, check_forward, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
def test_rms_norm_with_torchs_own_eps(dtype):
    """eps=None.  Rows near zero, where eps decides: it is float32's epsilon whatever the rows'
    type, in torch's module (to a few roundings of the type) and in this one (under the bound)."""
    dt = DTYPES[dtype]
    x = (torch.randn(6, 50, device="cuda") * 3e-4).to(dt)
    ours, theirs = nn.FlashRMSNorm(50, eps=None, device="cuda", dtype=dt), torch.nn.RMSNorm(50, device="cuda", dtype=dt)
    check_forward("y", ours(x), host(x), None, None, torch.finfo(torch.float32).eps, "rms")
    step = torch.finfo(dt).eps
    torch.testing.assert_close(ours(x), theirs(x), rtol=4 * step, atol=4 * step)
