"""The second float of the loss's log sums (CPU only): refusals of its array."""

import ctypes

import pytest

from precision_optimizer_state_amd import binding as B
from test_step_cpu import BASE, M, P, loss_args


@pytest.mark.parametrize("rest, rc, msg", [
    (0, B.FO_EINVAL, "rest is NULL"),
    (BASE + 7 * M + 2, B.FO_EINVAL, "aligned"),
    (BASE + 4 * M + 12, B.FO_EALIAS, "overlap"),         # lse
    (BASE + 64 * M, B.FO_EALIAS, "overlap"),             # the workspace
])
def test_refusals_of_the_forward_call(rest, rc, msg):
    assert B._load_step().fo_loss_forward_rest(ctypes.byref(loss_args()), P(rest), None) == rc
    assert msg in B.fo_last_error()


@pytest.mark.parametrize("rest, rc, msg", [
    (0, B.FO_EINVAL, "rest is NULL"),
    (BASE + 7 * M + 2, B.FO_EINVAL, "aligned"),
    (BASE + 8 * M + 16, B.FO_EALIAS, "overlap"),         # dx
    (BASE + 64 * M, B.FO_EALIAS, "overlap"),
])
def test_refusals_of_the_backward_call(rest, rc, msg):
    a = loss_args(dx=BASE + 8 * M)
    assert B._load_step().fo_loss_backward_rest(ctypes.byref(a), P(rest), None) == rc
    assert msg in B.fo_last_error()


def test_nothing_to_do():
    lib = B._load_step()
    a = loss_args(rows=0, reduction=0, x=None, weight=None, target=None, loss=None, lse=None, workspace=None, workspace_bytes=0)
    assert lib.fo_loss_forward_rest(ctypes.byref(a), None, None) == B.FO_OK
    assert lib.fo_loss_backward_rest(ctypes.byref(a), None, None) == B.FO_OK
    assert lib.fo_loss_forward_rest(None, P(BASE), None) == B.FO_EINVAL
    assert lib.fo_loss_backward_rest(None, P(BASE), None) == B.FO_EINVAL
