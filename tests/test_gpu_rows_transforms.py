"""Forward-mode derivatives and tracers meet the row operators on the GPU: a
tangent or a trace is refused; neither comes back without the operator's part."""

import pytest
import torch
import torch.autograd.forward_ad as fwAD

from precision_optimizer_state_amd import nn

pytestmark = pytest.mark.gpu


def calls(x, r, w, b):
    return {"dropout": lambda: nn.dropout(x, 0.5, 1), "layer_norm": lambda: nn.layer_norm(x, w, b),
            "rms_norm": lambda: nn.rms_norm(x, w), "join": lambda: nn.dropout_add_layer_norm(x, r, w, b, p=0.1)[1]}


OPS = ["dropout", "layer_norm", "rms_norm", "join"]


def arguments():
    return [torch.randn(4, 8, device="cuda"), torch.randn(4, 8, device="cuda"), torch.ones(8, device="cuda"),
            torch.zeros(8, device="cuda")]


@pytest.mark.parametrize("op", OPS)
def test_forward_mode_is_refused(op):
    args = arguments()
    plain = calls(*args)[op]()
    with fwAD.dual_level():
        dual = [fwAD.make_dual(args[0], torch.ones_like(args[0]))] + args[1:]
        with pytest.raises(NotImplementedError, match="forward-mode"):
            calls(*dual)[op]()
        assert torch.equal(calls(*args)[op](), plain)            # a plain call at the same level
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda t: calls(t, *args[1:])[op](), (args[0],), (args[0],))


@pytest.mark.parametrize("op", OPS)
def test_forward_mode_through_a_backward_pass_is_refused(op):
    args = arguments()
    args[0].requires_grad_(True)
    y = calls(*args)[op]()
    with fwAD.dual_level():
        dy = fwAD.make_dual(torch.ones_like(y), torch.ones_like(y))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            torch.autograd.grad(y, args[0], dy)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("pre_dispatch", [False, True])
def test_tracers_are_refused(op, pre_dispatch):
    from torch.fx.experimental.proxy_tensor import make_fx
    args = arguments()
    want = calls(*args)[op]()
    with pytest.raises(NotImplementedError, match="traced"):
        make_fx(lambda t: calls(t, *args[1:])[op](), pre_dispatch=pre_dispatch)(args[0])
    with pytest.raises(NotImplementedError, match="traced"):
        torch.jit.trace(lambda t: calls(t, *args[1:])[op](), args[0], check_trace=False)
    with pytest.raises(Exception):                                # fake tensors have no memory
        make_fx(lambda t: calls(t, *args[1:])[op](), tracing_mode="fake")(args[0])
    assert torch.equal(calls(*args)[op](), want)


@pytest.mark.parametrize("op", OPS)
def test_a_traced_backward_pass_is_refused(op):
    from torch.fx.experimental.proxy_tensor import make_fx
    args = arguments()
    args[0].requires_grad_(True)
    y = calls(*args)[op]()
    with pytest.raises(NotImplementedError, match="traced"):
        make_fx(lambda dy: torch.autograd.grad(y, args[0], dy, retain_graph=True)[0])(torch.ones_like(y))
    torch.autograd.grad(y, args[0], torch.ones_like(y))
