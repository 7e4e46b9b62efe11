"""Calls of the row operators that torch would have to see through, and cannot:
forward-mode derivatives and tracers.  They are refused before anything else is
looked at, so host tensors do here."""

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


OPS = ["dropout", "layer_norm", "rms_norm", "join_layer", "join_rms"]


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("pre_dispatch", [False, True])
def test_make_fx_is_refused(op, grad, pre_dispatch):
    from torch.fx.experimental.proxy_tensor import make_fx
    r, w, b = torch.randn(4, 8), torch.ones(8), torch.zeros(8)
    x = torch.randn(4, 8).requires_grad_(grad)
    with pytest.raises(NotImplementedError, match="traced"):
        make_fx(lambda t: calls(t, r, w, b)[op](), pre_dispatch=pre_dispatch)(x)


@pytest.mark.parametrize("op", OPS)
def test_jit_trace_is_refused(op):
    r, w, b = torch.randn(4, 8), torch.ones(8), torch.zeros(8)
    with pytest.raises(NotImplementedError, match="traced"):
        torch.jit.trace(lambda t: calls(t, r, w, b)[op](), torch.randn(4, 8), check_trace=False)


def test_other_modes_are_let_through():
    # a dispatch mode that only watches reaches the check of the device
    from torch.utils._python_dispatch import TorchDispatchMode

    class Watch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            return func(*args, **(kwargs or {}))

    with Watch(), pytest.raises(ValueError, match="GPU"):
        nn.rms_norm(torch.randn(4, 8))
    with pytest.raises(ValueError, match="GPU"):
        nn.rms_norm(torch.randn(4, 8))
