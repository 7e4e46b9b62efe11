"""Forward-mode derivatives of the row operators are refused before anything else
is looked at, so host tensors do here."""

import pytest
import torch
import torch.autograd.forward_ad as fwAD

from precision_optimizer_state_amd import nn


def calls(x, r, w, b):
    return {"dropout": lambda: nn.dropout(x, 0.5, 1), "layer_norm": lambda: nn.layer_norm(x, w, b),
            "rms_norm": lambda: nn.rms_norm(x, w), "join_layer": lambda: nn.dropout_add_layer_norm(x, r, w, b, p=0.1),
            "join_rms": lambda: nn.dropout_add_rms_norm(x, r, w)}


@pytest.mark.parametrize("op, which", [("dropout", 0), ("layer_norm", 0), ("layer_norm", 2), ("layer_norm", 3),
                                       ("rms_norm", 0), ("rms_norm", 2), ("join_layer", 0), ("join_layer", 1),
                                       ("join_layer", 3), ("join_rms", 1), ("join_rms", 2)])
@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused(op, which, grad):
    args = [torch.randn(4, 8), torch.randn(4, 8), torch.ones(8), torch.zeros(8)]
    with fwAD.dual_level():
        args[which] = fwAD.make_dual(args[which].requires_grad_(grad), torch.ones_like(args[which]))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            calls(*args)[op]()
        x = args[0]
        assert nn.dropout(x, 0.0, 1) is x
