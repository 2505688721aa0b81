"""The layer norm of finite rows whose elements differ from their mean by more than the largest
fp32 value: the outputs are of ordinary size, and so are the weight's gradients."""
import pytest
import torch

import _more_ref as M
import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops
from test_gpu_ops_layer_norm import check_forward, gen, rand

pytestmark = pytest.mark.gpu
E = R.E
WIDTHS = [8, 40, 515, 1001, 2048, 8192, 8200, 12289]


def far_apart(rows, width, dtype, seed):
    """Rows of +-(2.9 to 3.3)e38, one element in eight on the other side, so that the mean is some
    2.3e38 and the differences up to 5.6e38; the last row is an ordinary one."""
    g = gen(seed)
    x = 2.9e38 + torch.rand(rows, width, generator=g, device="cuda") * 0.4e38
    x[:, ::8] *= -1
    x[::2] *= -1
    x[-1] = torch.randn(width, generator=g, device="cuda")
    x = x.to(dtype)
    assert bool(torch.isfinite(x).all())
    d = (R.f64(x) - R.f64(x).mean(1, keepdim=True)).abs()
    assert bool((d[:-1].amax(1) > torch.finfo(torch.float32).max).all())
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", WIDTHS)
def test_forward(dtype, width):
    g = gen(width)
    x = far_apart(5, width, dtype, width)
    w, b = rand(g, width, dtype=dtype, std=0.2, shift=1.0), rand(g, width, dtype=dtype, std=0.3)
    r = check_forward(x, w, b, None, 1e-5)
    # the path with codes has the same output
    assert bool(torch.isfinite(check_forward(x, w, b, None, 1e-5, "e4m3").y).all())
    assert bool(torch.isfinite(r.y).all())
    # as the sum with a residual
    half = x * 0.5
    check_forward(half, w, b, half, 1e-5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", WIDTHS)
def test_backward(dtype, width):
    g = gen(width + 1)
    rows = 41
    s = far_apart(rows, width, dtype, width + 2)
    dy, w = rand(g, rows, width, dtype=dtype), rand(g, width, dtype=dtype, std=0.2, shift=1.0)
    x = R.f64(s)
    mean = x.mean(1)
    rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + 1e-5)
    mean, rstd = mean.float(), rstd.float()
    want = M.layer_norm_grad(R.f64(dy), x, R.f64(w), mean.double(), rstd.double(), None)
    dx, dw, db = ops.layer_norm_backward(dy, s, w, mean.cuda(), rstd.cuda(), weight_grad_dtype=torch.float32)
    # as for other rows: a lane adds up to 64 terms and joins 10 times, and ten roundings of a term;
    # here dx is below fp32's normal range before its rounding to the type, which may round it twice
    R.close(dx, want[0], want[0].abs() * R.u(dtype) * 1.01 + want[3] * 96 * E + R.sub(dtype) + R.sub(torch.float32), "dx")
    # under 260 additions of a column
    R.close(dw, want[1], want[1].abs() * E * 1.01 + want[4] * 260 * E, "dw")
    R.close(db, want[2], want[2].abs() * E * 1.01 + want[5] * 260 * E, "db")


def within(rows, width, dtype, seed):
    """One row a power of two, from deviations of 2^96 to 2^126, some far from zero."""
    g = gen(seed)
    e = torch.linspace(96, 126, rows, device="cuda").round()
    x = torch.rand(rows, width, generator=g, device="cuda") * 2 - 1
    x[::3] += 0.75
    x = (x * torch.exp2(e)[:, None]).to(dtype)
    assert bool(torch.isfinite(x).all())
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", [40, 1001, 8200, 40000])
def test_deviations_below_and_above_the_border(dtype, width):
    g = gen(width)
    x = within(31, width, dtype, width)
    w, b = rand(g, width, dtype=dtype, std=0.2, shift=1.0), rand(g, width, dtype=dtype, std=0.3)
    check_forward(x, w, b, None, 1e-5)
    check_forward(x, w, None, None, 0.0)
    dy = rand(g, 31, width, dtype=dtype)
    s = R.f64(x)
    mean = s.mean(1)
    rstd = 1 / torch.sqrt(((s - mean[:, None]) ** 2).mean(1))
    mean, rstd = mean.float(), rstd.float()
    want = M.layer_norm_grad(R.f64(dy), s, R.f64(w), mean.double(), rstd.double(), None)
    dx, dw, _ = ops.layer_norm_backward(dy, x, w, mean.cuda(), rstd.cuda(), weight_grad_dtype=torch.float32)
    # as above
    R.close(dx, want[0], want[0].abs() * R.u(dtype) * 1.01 + want[3] * 96 * E + R.sub(dtype) + R.sub(torch.float32), "dx")
    R.close(dw, want[1], want[1].abs() * E * 1.01 + want[4] * 260 * E, "dw")
