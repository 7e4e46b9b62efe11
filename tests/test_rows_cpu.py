"""Argument checks of the row operators (CPU only: every call here fails, or has
nothing to do, before any GPU work)."""

import ctypes

import pytest
import torch

from precision_optimizer_state_amd import binding as B
from precision_optimizer_state_amd import nn

P = ctypes.c_void_p
BASE = 1 << 24


def key(p=0.0, state=None):
    return B.DropoutKey(p, 1, 2, state)


def fwd(**kw):
    a = dict(x=BASE, residual=None, weight=None, bias=None, h=None, y=BASE + (1 << 20), mean=None, rstd=None,
             rows=4, cols=64, x_ld=64, residual_ld=64, eps=1e-5, drop=key(), dtype=B.FO_BF16, wdtype=B.FO_F32,
             kind=B.FO_LAYER_NORM, reserved=0)
    a.update(kw)
    return B.load().fo_norm_forward(ctypes.byref(B.NormFwd(**a)), None)


def bwd(**kw):
    m = 1 << 20
    a = dict(dy=BASE, dh=None, h=BASE + m, weight=None, mean=BASE + 2 * m, rstd=BASE + 3 * m, d=BASE + 4 * m, dx=None,
             dweight=None, dbias=None, workspace=None, workspace_bytes=0, rows=4, cols=64, dy_ld=64, dh_ld=64, h_ld=64,
             drop=key(), dtype=B.FO_BF16, wdtype=B.FO_F32, kind=B.FO_LAYER_NORM, reserved=0)
    a.update(kw)
    return B.load().fo_norm_backward(ctypes.byref(B.NormBwd(**a)), None)


def drop(x=BASE, ld=64, y=BASE + (1 << 20), rows=4, cols=64, dtype=B.FO_BF16, k=None):
    return B.load().fo_dropout(P(x), ld, P(y), rows, cols, dtype, ctypes.byref(k or key(0.5)), None)


def test_struct_layouts():
    assert ctypes.sizeof(B.DropoutKey) == 32
    assert ctypes.sizeof(B.NormFwd) == 8 * 8 + 4 * 8 + 8 + 32 + 16
    assert ctypes.sizeof(B.NormBwd) == 11 * 8 + 6 * 8 + 32 + 16


@pytest.mark.parametrize("kw, rc, msg", [
    (dict(x=None), B.FO_EINVAL, "x is NULL"),
    (dict(y=None), B.FO_EINVAL, "y is NULL"),
    (dict(x=BASE + 1), B.FO_EINVAL, "aligned"),
    (dict(x=BASE + 2, dtype=B.FO_F32), B.FO_EINVAL, "aligned"),
    (dict(cols=0), B.FO_EINVAL, "cols"),
    (dict(cols=(1 << 26) + 1, x_ld=1 << 27), B.FO_EINVAL, "cols"),
    (dict(rows=-1), B.FO_EINVAL, "rows"),
    (dict(rows=(1 << 40) + 1), B.FO_EINVAL, "rows"),
    (dict(x_ld=-1), B.FO_EINVAL, "stride"),
    (dict(x_ld=(1 << 62)), B.FO_EINVAL, "address space"),
    (dict(rows=1 << 40, cols=1 << 26, x_ld=0), B.FO_EINVAL, "address space"),
    (dict(dtype=3), B.FO_EINVAL, "element type"),
    (dict(wdtype=-1), B.FO_EINVAL, "element type"),
    (dict(kind=2), B.FO_EINVAL, "kind"),
    (dict(eps=-1e-5), B.FO_EINVAL, "eps"),
    (dict(eps=float("nan")), B.FO_EINVAL, "eps"),
    (dict(eps=float("inf")), B.FO_EINVAL, "eps"),
    (dict(drop=key(0.1)), B.FO_EINVAL, "residual"),
    (dict(h=BASE + (1 << 21)), B.FO_EINVAL, "residual"),
    (dict(residual=BASE + (1 << 21)), B.FO_EINVAL, "h is NULL"),
    (dict(residual=BASE + (1 << 21), h=BASE + (1 << 22), drop=key(1.5)), B.FO_EINVAL, "probability"),
    (dict(residual=BASE + (1 << 21), h=BASE + (1 << 22), drop=key(float("nan"))), B.FO_EINVAL, "probability"),
    (dict(residual=BASE + (1 << 21), h=BASE + (1 << 22), drop=key(0.5, BASE + 4)), B.FO_EINVAL, "state"),
    (dict(kind=B.FO_RMS_NORM, bias=BASE + (1 << 21)), B.FO_EINVAL, "RMS"),
    (dict(kind=B.FO_RMS_NORM, mean=BASE + (1 << 21)), B.FO_EINVAL, "RMS"),
    (dict(y=BASE), B.FO_EALIAS, "overlap"),
    (dict(y=BASE + 3 * 128 + 64), B.FO_EALIAS, "overlap"),
    (dict(y=BASE + 1000, x_ld=300), B.FO_EALIAS, "overlap"),
    (dict(mean=BASE + (1 << 20) + 16), B.FO_EALIAS, "overlap"),
    (dict(residual=BASE + (1 << 21), h=BASE + (1 << 21)), B.FO_EALIAS, "overlap"),
])
def test_forward_refusals(kw, rc, msg):
    assert fwd(**kw) == rc
    assert msg in B.fo_last_error()


@pytest.mark.parametrize("kw, rc, msg", [
    (dict(dy=None), B.FO_EINVAL, "dy is NULL"),
    (dict(h=None), B.FO_EINVAL, "h is NULL"),
    (dict(mean=None), B.FO_EINVAL, "mean is NULL"),
    (dict(rstd=None), B.FO_EINVAL, "rstd is NULL"),
    (dict(rstd=BASE + 2), B.FO_EINVAL, "aligned"),
    (dict(dy_ld=-64), B.FO_EINVAL, "stride"),
    (dict(dx=BASE + (1 << 23)), B.FO_EINVAL, "dropout"),
    (dict(kind=B.FO_RMS_NORM), B.FO_EINVAL, "RMS"),
    (dict(kind=B.FO_RMS_NORM, mean=None, dbias=BASE + (1 << 23)), B.FO_EINVAL, "RMS"),
    (dict(dweight=BASE + (1 << 23)), B.FO_EINVAL, "workspace"),
    (dict(dweight=BASE + (1 << 23), workspace=BASE + (1 << 22) + (1 << 23), workspace_bytes=100), B.FO_EINVAL,
     "workspace"),
    (dict(dweight=BASE + (1 << 23), workspace=BASE + 8 + (1 << 24), workspace_bytes=1 << 20), B.FO_EINVAL,
     "workspace is not 16-byte"),
    (dict(dbias=BASE + (1 << 23), workspace=BASE, workspace_bytes=1 << 20), B.FO_EALIAS, "overlap"),
    (dict(d=BASE), B.FO_EALIAS, "overlap"),
    (dict(dweight=BASE + (1 << 23), dbias=BASE + (1 << 23) + 16, workspace=BASE + (1 << 24),
          workspace_bytes=1 << 20), B.FO_EALIAS, "overlap"),
    (dict(drop=key(-0.1)), B.FO_EINVAL, "probability"),
    (dict(cols=0), B.FO_EINVAL, "cols"),
])
def test_backward_refusals(kw, rc, msg):
    assert bwd(**kw) == rc
    assert msg in B.fo_last_error()


@pytest.mark.parametrize("kw, rc, msg", [
    (dict(x=0), B.FO_EINVAL, "x is NULL"),
    (dict(y=0), B.FO_EINVAL, "y is NULL"),
    (dict(rows=-1), B.FO_EINVAL, "rows"),
    (dict(cols=-1), B.FO_EINVAL, "cols"),
    (dict(rows=0, cols=-1), B.FO_EINVAL, "negative"),
    (dict(dtype=7), B.FO_EINVAL, "element type"),
    (dict(k=B.DropoutKey(2.0, 0, 0, None)), B.FO_EINVAL, "probability"),
    (dict(y=BASE), B.FO_EALIAS, "overlap"),
    (dict(y=BASE + 128), B.FO_EALIAS, "overlap"),
])
def test_dropout_refusals(kw, rc, msg):
    assert drop(**kw) == rc
    assert msg in B.fo_last_error()
    assert B.load().fo_dropout(P(BASE), 64, P(BASE), 4, 64, 0, None, None) == B.FO_EINVAL


def test_nothing_to_do():
    assert drop(rows=0) == B.FO_OK and drop(cols=0) == B.FO_OK
    assert fwd(rows=0) == B.FO_OK and fwd(rows=0, x=None, y=None) == B.FO_OK
    assert bwd(rows=0) == B.FO_OK
    assert B.fo_last_error() == ""


def test_workspace_query():
    assert B.fo_norm_backward_workspace(0, 768) >= 0
    small, large = B.fo_norm_backward_workspace(10, 768), B.fo_norm_backward_workspace(1 << 20, 768)
    assert 0 < small <= large <= 64 << 20
    with pytest.raises(B.FoError):
        B.fo_norm_backward_workspace(-1, 8)
    with pytest.raises(B.FoError):
        B.fo_norm_backward_workspace(8, 0)
    assert B.load().fo_norm_backward_workspace(8, 8, None) == B.FO_EINVAL


def test_host_tensors_are_refused():
    x, w = torch.zeros(4, 8), torch.ones(8)
    for call in (lambda: nn.layer_norm(x, w), lambda: nn.rms_norm(x), lambda: nn.dropout(x, 0.5, 1),
                 lambda: nn.dropout_add_layer_norm(x, x), lambda: B.fo_dropout(x, x, B.dropout_key(0.1, 0))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_a_library_without_the_row_operators_still_loads(monkeypatch):
    class Old:
        pass
    monkeypatch.setattr(B, "_lib", Old())
    with pytest.raises(ImportError, match="row operators"):
        B._load_rows()


def test_counter():
    c = nn.DropoutCounter(5, 10)
    assert c.next() == {"seed": 5, "offset": 10, "state": None} and c.next()["offset"] == 11
    d = nn.DropoutCounter(0)
    d.load_state_dict(c.state_dict())
    assert d.next() == {"seed": 5, "offset": 12, "state": None}
    with pytest.raises(ValueError):
        c.advance()
    on_device = nn.DropoutCounter(5, device="cpu")
    with pytest.raises(ValueError):
        on_device.load_state_dict(c.state_dict())
    on_device.advance()
    saved = on_device.state_dict()
    again = nn.DropoutCounter(0, device="cpu")
    again.load_state_dict(saved)
    assert again.state.tolist() == [0, 1 << 32] and again.seed == 5
    with pytest.raises(ValueError, match="probability"):
        nn.FlashDropout(1.2, c)
