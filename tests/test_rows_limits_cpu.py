"""Size limits of fo_dropout, without a GPU: calls whose arrays overlap fail on
that, and so show that their sizes were accepted."""

import ctypes

import pytest

from precision_optimizer_state_amd import binding as B

BASE = 1 << 24


@pytest.mark.parametrize("rows, cols, dtype, rc, msg", [
    (1, 1 << 26, B.FO_BF16, B.FO_EALIAS, "overlap"),
    (1, (1 << 26) + 1, B.FO_F32, B.FO_EALIAS, "overlap"),
    (3, (1 << 33) + 5, B.FO_BF16, B.FO_EALIAS, "overlap"),
    (1, 1 << 40, B.FO_F32, B.FO_EALIAS, "overlap"),
    (1, (1 << 40) + 1, B.FO_F32, B.FO_EINVAL, "cols"),
    (1 << 40, 1 << 40, B.FO_F32, B.FO_EINVAL, "address space"),
    ((1 << 40) + 1, 8, B.FO_F32, B.FO_EINVAL, "rows"),
])
def test_dropout_sizes(rows, cols, dtype, rc, msg):
    P = ctypes.c_void_p
    key = B.DropoutKey(0.5, 1, 2, None)
    assert B.load().fo_dropout(P(BASE), cols, P(BASE + 64), rows, cols, dtype, ctypes.byref(key), None) == rc
    assert msg in B.fo_last_error()
