"""Argument checks of gradient clipping, linear cross entropy and the gated block (CPU
only: every call here fails, or has nothing to do, before any GPU work)."""

import ctypes
import math

import pytest
import torch

from precision_optimizer_state_amd import FlashAdamW, binding as B, grads, nn

P = ctypes.c_void_p
BASE = 1 << 24
M = 1 << 20


def test_struct_layouts():
    assert ctypes.sizeof(B.Grad) == 32
    assert ctypes.sizeof(B.Loss) == 10 * 8 + 8 + 7 * 8 + 8 + 8
    assert ctypes.sizeof(B.Gated) == 11 * 8 + 8 + 7 * 8 + 8


# ---------------------------------------------------------------------------
# clipping
# ---------------------------------------------------------------------------
def clip(rows, order=B.FO_NORM_2, max_norm=1.0, norm=BASE - 4096, ws=BASE - 65536, nbytes=1 << 15, count=None):
    lib = B._load_step()
    arr = (B.Grad * max(1, len(rows)))(*[B.Grad(*r) for r in rows])
    n = len(rows) if count is None else count
    if max_norm is None:
        return lib.fo_grad_norm(arr, n, order, P(norm), P(ws), nbytes, None)
    return lib.fo_grad_clip(arr, n, order, max_norm, P(norm), P(ws), nbytes, None)


ROW = (BASE, BASE, 64, B.FO_BF16, B.FO_BF16)


@pytest.mark.parametrize("rows, kw, rc, msg", [
    ([ROW], dict(order=3), B.FO_EINVAL, "order"),
    ([ROW], dict(order=-1), B.FO_EINVAL, "order"),
    ([ROW], dict(count=-1), B.FO_EINVAL, "count"),
    ([ROW], dict(count=(1 << 17) + 1), B.FO_EINVAL, "count"),
    ([ROW], dict(norm=0), B.FO_EINVAL, "norm"),
    ([ROW], dict(norm=BASE - 4094), B.FO_EINVAL, "norm"),
    ([ROW], dict(ws=0), B.FO_EINVAL, "workspace"),
    ([ROW], dict(ws=BASE - 65536 + 16), B.FO_EINVAL, "workspace"),
    ([ROW], dict(nbytes=100), B.FO_EINVAL, "workspace"),
    ([ROW], dict(max_norm=-1.0), B.FO_EINVAL, "max_norm"),
    ([ROW], dict(max_norm=math.nan), B.FO_EINVAL, "max_norm"),
    ([(BASE, BASE, -1, 0, 0)], {}, B.FO_EINVAL, "n = -1"),
    ([(BASE, BASE, 64, 3, 0)], {}, B.FO_EINVAL, "element type"),
    ([(BASE, BASE, 64, 0, -1)], {}, B.FO_EINVAL, "element type"),
    ([(0, BASE, 64, 0, 0)], {}, B.FO_EINVAL, "grad is NULL"),
    ([(BASE + 1, BASE + 1, 64, 0, 0)], {}, B.FO_EINVAL, "misaligned"),
    ([(BASE, 0, 64, 0, 0)], {}, B.FO_EINVAL, "out is NULL"),
    ([(BASE, BASE, 64, B.FO_BF16, B.FO_FP16)], {}, B.FO_EINVAL, "another type"),
    ([((1 << 64) - 64, (1 << 64) - 64, 64, 0, 0)], {}, B.FO_EINVAL, "address space"),
    # overlaps: a tensor twice, an output on another's input, two outputs, the scratch arrays
    ([ROW, ROW], {}, B.FO_EALIAS, "overlap"),
    ([ROW, (BASE + 64, BASE + 64, 64, 0, 0)], {}, B.FO_EALIAS, "overlap"),
    ([(BASE, BASE + M, 64, 0, 0), (BASE + M + 126, BASE + 2 * M, 64, 0, 0)], {}, B.FO_EALIAS, "overlap"),
    ([(BASE, BASE + M, 64, 0, 2), (BASE + 4 * M, BASE + M + 255 - 3, 64, 0, 2)], {}, B.FO_EALIAS, "overlap"),
    ([(BASE, BASE + 2, 64, 0, 0)], {}, B.FO_EALIAS, "overlap"),
    ([ROW], dict(norm=BASE + 64), B.FO_EALIAS, "overlap"),
    ([ROW], dict(ws=BASE - 256), B.FO_EALIAS, "overlap"),
    ([ROW], dict(norm=BASE - 65536 + 128), B.FO_EALIAS, "overlap"),
    ([ROW], dict(norm=BASE + 4, max_norm=None), B.FO_EALIAS, "overlap"),
])
def test_clip_refusals(rows, kw, rc, msg):
    assert clip(rows, **kw) == rc
    assert msg in B.fo_last_error()


def test_clip_overlaps_that_are_none():
    """Arrays side by side, in any order, and inputs that only the norm reads twice:
    the call then fails at the device that is not there, not at its arguments."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not a GPU's")
    for rows in ([(BASE + 128, BASE + 128, 64, 0, 0), ROW], [(BASE, BASE + M, 64, 0, 0), (BASE, BASE + M + 128, 64, 0, 0)]):
        assert clip(rows) == B.FO_EHIP
    assert clip([ROW, ROW], max_norm=None) == B.FO_EHIP


def test_grad_workspace():
    lib = B._load_step()
    assert lib.fo_grad_workspace(None) == B.FO_EINVAL
    assert 0 < B.fo_grad_workspace() <= 1 << 15


def test_python_refuses_orders_bounds_and_host_tensors():
    g = torch.ones(8)
    for norm_type in (0, 3, -1, "x", math.nan, -math.inf):
        with pytest.raises(ValueError):
            grads.grad_norm([g], norm_type)
    for bound in (-1.0, math.nan):
        with pytest.raises(ValueError, match="max_norm"):
            grads.clip_grads([g], bound)
    with pytest.raises(ValueError, match="GPU"):
        grads.grad_norm([g])
    with pytest.raises(ValueError, match="GPU"):
        grads.clip_grads([g], 1.0)
    p = torch.nn.Parameter(torch.ones(8))
    p.grad = g
    with pytest.raises(ValueError, match="GPU"):
        grads.clip_grad_norm_([p], 1.0)
    with pytest.raises(ValueError, match="tensors"):
        grads.clip_grads([g], 1.0, out=[])
    with pytest.raises(ValueError, match="GPU"):
        B.fo_grad_norm([g], torch.ones(1))


def test_optimizer_with_gradient_release_refuses():
    opt = FlashAdamW.__new__(FlashAdamW)
    opt.grad_release, opt.param_groups = True, []
    with pytest.raises(RuntimeError, match="grad_release"):
        opt.clip_grad_norm_(1.0)


# ---------------------------------------------------------------------------
# linear cross entropy
# ---------------------------------------------------------------------------
def loss_args(**kw):
    a = dict(x=BASE, weight=BASE + M, target=BASE + 2 * M, loss=BASE + 3 * M, lse=BASE + 4 * M, count=BASE + 5 * M,
             dloss=BASE + 6 * M, dx=None, dweight=None, workspace=BASE + 64 * M, workspace_bytes=64 * M,
             rows=4, cols=64, vocab=100, x_ld=64, weight_ld=64, dloss_ld=1, ignore_index=-100, smoothing=0.0,
             dtype=B.FO_BF16, reduction=1)
    a.update(kw)
    return B.Loss(**a)


@pytest.mark.parametrize("kw, rc, msg", [
    (dict(dtype=3), B.FO_EINVAL, "element type"),
    (dict(reduction=3), B.FO_EINVAL, "reduction"),
    (dict(reduction=-1), B.FO_EINVAL, "reduction"),
    (dict(rows=-1), B.FO_EINVAL, "rows"),
    (dict(rows=(1 << 21) + 1), B.FO_EINVAL, "rows"),
    (dict(cols=0), B.FO_EINVAL, "cols"),
    (dict(cols=(1 << 20) + 1), B.FO_EINVAL, "cols"),
    (dict(vocab=0), B.FO_EINVAL, "vocab"),
    (dict(vocab=(1 << 24) + 1), B.FO_EINVAL, "vocab"),
    (dict(rows=1 << 20, vocab=1 << 17), B.FO_EINVAL, "2^36"),
    (dict(cols=1 << 18, vocab=1 << 20), B.FO_EINVAL, "2^36"),
    (dict(smoothing=-0.1), B.FO_EINVAL, "smoothing"),
    (dict(smoothing=1.1), B.FO_EINVAL, "smoothing"),
    (dict(smoothing=math.nan), B.FO_EINVAL, "smoothing"),
    (dict(x=None), B.FO_EINVAL, "x is NULL"),
    (dict(weight=None), B.FO_EINVAL, "weight is NULL"),
    (dict(target=None), B.FO_EINVAL, "target is NULL"),
    (dict(target=BASE + 2 * M + 4), B.FO_EINVAL, "aligned"),
    (dict(x_ld=-1), B.FO_EINVAL, "stride"),
    (dict(lse=None), B.FO_EINVAL, "lse is NULL"),
])
def test_loss_refusals_of_both_ways(kw, rc, msg):
    lib = B._load_step()
    for call in (lib.fo_loss_forward, lib.fo_loss_backward):
        assert call(ctypes.byref(loss_args(**kw)), None) == rc
        assert msg in B.fo_last_error()


@pytest.mark.parametrize("kw, rc, msg", [
    (dict(loss=None), B.FO_EINVAL, "loss is NULL"),
    (dict(count=None), B.FO_EINVAL, "count is NULL"),
    (dict(workspace_bytes=16), B.FO_EINVAL, "workspace"),
    (dict(workspace=BASE + 64 * M + 128), B.FO_EINVAL, "256-byte"),
    (dict(loss=BASE + 128), B.FO_EALIAS, "overlap"),
    (dict(lse=BASE + 3 * M), B.FO_EALIAS, "overlap"),
    (dict(workspace=BASE), B.FO_EALIAS, "overlap"),
])
def test_loss_forward_refusals(kw, rc, msg):
    assert B._load_step().fo_loss_forward(ctypes.byref(loss_args(**kw)), None) == rc
    assert msg in B.fo_last_error()


@pytest.mark.parametrize("kw, rc, msg", [
    (dict(dx=BASE + 8 * M, dloss=None), B.FO_EINVAL, "dloss is NULL"),
    (dict(dx=BASE + 8 * M, count=None), B.FO_EINVAL, "count is NULL"),
    (dict(dx=BASE), B.FO_EALIAS, "overlap"),
    (dict(dweight=BASE + M + 64), B.FO_EALIAS, "overlap"),
    (dict(dx=BASE + 8 * M, dweight=BASE + 8 * M), B.FO_EALIAS, "overlap"),
    (dict(dx=BASE + 8 * M, workspace_bytes=0), B.FO_EINVAL, "workspace"),
    (dict(dx=BASE + 8 * M + 1), B.FO_EINVAL, "aligned"),
])
def test_loss_backward_refusals(kw, rc, msg):
    assert B._load_step().fo_loss_backward(ctypes.byref(loss_args(**kw)), None) == rc
    assert msg in B.fo_last_error()


def test_loss_with_nothing_to_do():
    lib = B._load_step()
    assert lib.fo_loss_forward(ctypes.byref(loss_args(rows=0, reduction=0, x=None, weight=None, target=None, loss=None,
                                                      lse=None, workspace=None, workspace_bytes=0)), None) == B.FO_OK
    assert lib.fo_loss_backward(ctypes.byref(loss_args(workspace=None, workspace_bytes=0)), None) == B.FO_OK
    assert lib.fo_loss_forward(None, None) == B.FO_EINVAL and lib.fo_loss_backward(None, None) == B.FO_EINVAL
    n = ctypes.c_int64(7)
    assert lib.fo_loss_backward_workspace(ctypes.byref(loss_args(rows=0)), ctypes.byref(n)) == B.FO_OK and n.value == 0
    assert lib.fo_loss_forward_workspace(ctypes.byref(loss_args()), None) == B.FO_EINVAL


def test_python_loss_refusals():
    x, w, t = torch.zeros(4, 8), torch.zeros(10, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="reduction"):
        nn.linear_cross_entropy(x, w, t, reduction="max")
    for s in (-0.1, 1.5, math.nan):
        with pytest.raises(ValueError, match="label_smoothing"):
            nn.linear_cross_entropy(x, w, t, label_smoothing=s)
    with pytest.raises(ValueError, match="GPU"):
        nn.linear_cross_entropy(x, w, t)
    with pytest.raises(ValueError, match="last dimension"):
        nn.linear_cross_entropy(torch.zeros(()), w, t)
    with pytest.raises(ValueError, match="GPU"):
        B.fo_loss_forward(x, w, t, torch.zeros(1), torch.zeros(4), torch.zeros(1))
    with pytest.raises(TypeError):
        nn.linear_cross_entropy(x, w, None)


# ---------------------------------------------------------------------------
# the gated block
# ---------------------------------------------------------------------------
def gated_args(**kw):
    a = dict(x=BASE, gate=BASE + M, up=BASE + 2 * M, y=BASE + 3 * M, g=BASE + 4 * M, u=BASE + 5 * M, dy=BASE + 6 * M,
             dx=None, dgate=None, dup=None, workspace=BASE + 64 * M, workspace_bytes=64 * M, rows=4, cols=64, features=96,
             x_ld=64, gate_ld=64, up_ld=64, dy_ld=96, dtype=B.FO_BF16, activation=0)
    a.update(kw)
    return B.Gated(**a)


@pytest.mark.parametrize("kw, rc, msg", [
    (dict(dtype=-1), B.FO_EINVAL, "element type"),
    (dict(activation=3), B.FO_EINVAL, "activation"),
    (dict(rows=-1), B.FO_EINVAL, "rows"),
    (dict(cols=0), B.FO_EINVAL, "cols"),
    (dict(features=0), B.FO_EINVAL, "features"),
    (dict(features=(1 << 20) + 1), B.FO_EINVAL, "features"),
    (dict(cols=1 << 18, features=1 << 19), B.FO_EINVAL, "2^36"),
    (dict(x=None), B.FO_EINVAL, "x is NULL"),
    (dict(gate=None), B.FO_EINVAL, "gate is NULL"),
    (dict(up=None), B.FO_EINVAL, "up is NULL"),
    (dict(g=None), B.FO_EINVAL, "together"),
    (dict(gate_ld=-2), B.FO_EINVAL, "stride"),
])
def test_gated_refusals_of_both_ways(kw, rc, msg):
    lib = B._load_step()
    for call in (lib.fo_gated_forward, lib.fo_gated_backward):
        assert call(ctypes.byref(gated_args(dx=BASE + 8 * M, **kw)), None) == rc
        assert msg in B.fo_last_error()


@pytest.mark.parametrize("way, kw, rc, msg", [
    ("forward", dict(y=None), B.FO_EINVAL, "y is NULL"),
    ("forward", dict(y=BASE + M), B.FO_EALIAS, "overlap"),
    ("forward", dict(g=BASE + 5 * M), B.FO_EALIAS, "overlap"),
    ("forward", dict(cols=63, x_ld=63, gate_ld=63, up_ld=63, workspace=None), B.FO_EINVAL, "workspace"),
    ("backward", dict(dx=BASE + 8 * M, g=None, u=None), B.FO_EINVAL, "g is NULL"),
    ("backward", dict(dx=BASE + 8 * M, dy=None), B.FO_EINVAL, "dy is NULL"),
    ("backward", dict(dx=BASE + 4 * M), B.FO_EALIAS, "overlap"),
    ("backward", dict(dgate=BASE + 8 * M, dup=BASE + 8 * M + 64), B.FO_EALIAS, "overlap"),
    ("backward", dict(dup=BASE + 8 * M, workspace_bytes=1), B.FO_EINVAL, "workspace"),
])
def test_gated_refusals(way, kw, rc, msg):
    assert getattr(B._load_step(), "fo_gated_" + way)(ctypes.byref(gated_args(**kw)), None) == rc
    assert msg in B.fo_last_error()


def test_gated_with_nothing_to_do():
    lib = B._load_step()
    assert lib.fo_gated_forward(ctypes.byref(gated_args(rows=0, workspace=None)), None) == B.FO_OK
    assert lib.fo_gated_backward(ctypes.byref(gated_args(workspace=None)), None) == B.FO_OK
    assert lib.fo_gated_forward(None, None) == B.FO_EINVAL and lib.fo_gated_backward(None, None) == B.FO_EINVAL


def test_python_gated_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(10, 8)
    with pytest.raises(ValueError, match="activation"):
        nn.gated_linear(x, w, w, "tanh")
    with pytest.raises(ValueError, match="GPU"):
        nn.gated_linear(x, w, w)
    with pytest.raises(ValueError, match="GPU"):
        B.fo_gated_forward(x, w, w, torch.zeros(4, 10))
