"""The float32 sums over very many very long rows stay short chains."""

import numpy as np
import pytest
import torch

from precision_optimizer_state_amd import binding as B
from rows_helpers import U, check, col_depth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [200_003, 1037])
def test_weight_gradients_over_many_long_rows(rows):
    """One row of h and dy repeated (stride 0): the sums are known, and terms of one value a
    column make rounding errors of one sign, the worst a chain of additions can do."""
    cols = 262_144 + 264
    rng = np.random.default_rng(rows)
    h, dy = (rng.uniform(0.5, 1.0, cols).astype(np.float32) for _ in range(2))
    mean, rstd = np.float32(0.25), np.float32(1.5)
    hg, dyg = (torch.from_numpy(t).cuda().expand(rows, cols) for t in (h, dy))
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    B.fo_norm_backward(dyg, hg, torch.full((rows,), float(rstd), device="cuda"), "layer",
                       torch.full((rows,), float(mean), device="cuda"), dweight_out=dw, dbias_out=db)
    u = (h.astype(np.float64) - mean) * rstd
    # each term rounds h - mean, its product with rstd and the product with dy
    check("dbias", db, rows * dy.astype(np.float64), torch.float32, U * col_depth(rows) * rows * dy)
    check("dweight", dw, rows * dy * u, torch.float32, U * (col_depth(rows) + 4) * rows * dy * u)
