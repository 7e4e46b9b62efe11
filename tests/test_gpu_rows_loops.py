"""Norms whose backward kernels walk over several rows each, at the widths that
take the widest teams of lanes, two chunks per lane or the kernels of long rows;
row counts are no multiple of a turn.  Against the float64 oracle under the
bounds of rows_helpers.py."""

import pytest

from test_gpu_rows import run_norm

pytestmark = pytest.mark.gpu


# 256 workgroups take 2 rows of up to 4096 columns at a time, and one row of more
@pytest.mark.parametrize("kind, rows, cols, dtype, wdtype, join, p", [
    ("rms", 1601, 4096, "bf16", "bf16", False, 0.0),
    ("layer", 1601, 4095, "f32", "f32", False, 0.0),
    ("layer", 1601, 4095, "bf16", "f32", True, 0.1),
    ("rms", 1601, 4096, "f32", "f32", True, 0.3),
    ("layer", 801, 8192, "bf16", "bf16", True, 0.1),
    ("rms", 801, 8191, "fp16", "fp16", True, 0.0),
    ("layer", 801, 8191, "f32", "f32", False, 0.0),
    # two chunks per lane
    ("layer", 801, 16384, "bf16", "bf16", False, 0.0),
    ("rms", 801, 16383, "bf16", "bf16", True, 0.0),
    ("layer", 801, 16383, "fp16", "f32", True, 0.0),
    # long rows: the column kernel takes 8 rows of 43, 32 and 25 ranges of rows at a time
    ("layer", 801, 12000, "f32", "f32", False, 0.0),
    ("rms", 801, 16384, "bf16", "bf16", True, 0.2),
    ("layer", 801, 20000, "bf16", "bf16", True, 0.1),
])
def test_rows_of_several_turns(kind, rows, cols, dtype, wdtype, join, p):
    run_norm(kind, rows, cols, dtype, wdtype, join=join, p=p)
