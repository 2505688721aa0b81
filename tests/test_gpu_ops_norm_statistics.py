"""The norm's statistics for rows of any magnitude."""
import pytest
import torch

import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops

from test_gpu_ops_embed import DEV, TYPES, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [1, 3, 8, 40, 512, 1031, 8192, 20001])
def test_rstd_is_rounded_once(dtype, width):
    """Squares and their sum in fp64: rstd is off by its one rounding (and a part in 2^40)."""
    x = rows(300 if width < 2000 else 5, width, dtype, 1)
    rstd = R.norm(R.f64(x), torch.ones(width, dtype=torch.float64), 1e-6)[1]
    got = ops.norm(x, torch.ones(width, dtype=dtype, device=DEV), eps=1e-6).rstd
    R.close(got, rstd, rstd * R.E * (1 + 2.0 ** -16), "rstd")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("power", [-90, -70, 63, 64, 100, 120])
def test_rows_of_any_magnitude(dtype, power):
    """Finite rows whose squares leave fp32 are normalised like any other."""
    x = (rows(5, 200, torch.float32, 1) * 2.0 ** power).to(dtype)
    w = torch.ones(200, dtype=dtype, device=DEV)
    eps = 0.0 if power < 0 else 1e-6
    out = ops.norm(x, w, eps=eps, code="e4m3", group=32)
    y, rstd = R.norm(R.f64(x), R.f64(w), eps)
    R.close(out.rstd, rstd, rstd * R.E * (1 + 2.0 ** -16), "rstd")
    R.close(out.y, y, R.rounded(y, dtype, 3), "y")
