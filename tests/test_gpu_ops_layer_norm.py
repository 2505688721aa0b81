"""The layer norm and its gradient against float64: values, codes and scales, odd widths, strides,
misaligned views, means far above the deviations, values that are not finite, empty batches,
wide rows, offsets past 32 bits, side streams and graphs."""
import pytest
import torch

import _more_ref as M
import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops

pytestmark = pytest.mark.gpu
E = R.E
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def rand(g, *shape, dtype=torch.float32, std=1.0, shift=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + shift).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def check_forward(x, w, b, residual, eps, code=None, group=None, want_y=True):
    r = ops.layer_norm(x, w, b, residual=residual, eps=eps, code=code, group=group, want_y=want_y)
    s = R.f64(x)
    if residual is not None:
        R.close(r.sum, s + R.f64(residual), R.rounded(s + R.f64(residual), x.dtype, 1), "sum")
        s = R.f64(r.sum)
    else:
        assert r.sum is x
    y, mean, rstd, size = M.layer_norm(s, R.f64(w), R.f64(b) if b is not None else None, eps)
    # the sum in fp64 is off by 2^-52 of its magnitudes for each addition, far below the rounding
    R.close(r.mean, mean, R.rounded(mean, torch.float32) + s.abs().mean(1) * 2.0 ** -38, "mean")
    R.close(r.rstd, rstd, R.rounded(rstd, torch.float32), "rstd")
    if want_y:
        # six roundings of the product and the sum, rstd's among them, and one to the type
        R.close(r.y, y, y.abs() * R.u(x.dtype) * 1.01 + size * 8 * E + R.sub(x.dtype), "y")
    if code == "e2m1":
        want, byte = M.pack4(y)
        got, gbyte = M.read4(ops.Codes4(r.codes, r.scales, x.shape[1]))
        assert torch.equal(gbyte, byte) and torch.equal(got, want)
    elif code:
        want, byte = exact8(y, code, group or 128)
        assert torch.equal(R.byte_of(r.scales), byte)
        assert torch.equal(r.codes.cpu().float(), want.float())
    else:
        assert r.codes is None and r.scales is None
    return r


def exact8(y, code, group):
    """pack of float64 values in one rounding: (codes' values, scale bytes)"""
    top, bits, low = {"e4m3": (1.75 * 2 ** 8, 3, -6), "e5m2": (1.75 * 2 ** 15, 2, -14)}[code]
    rows, d = y.shape
    n = -(-d // group)
    p = torch.zeros(rows, n * group, dtype=torch.float64)
    p[:, :d] = y
    p = p.view(rows, n, group)
    amax = p.abs().amax(2)
    e = torch.full_like(amax, -127)
    for k in range(-126, 128):
        e = torch.where(amax > top * 2.0 ** (k - 1), torch.full_like(e, k), e)
    q = p * torch.exp2(-e)[:, :, None]
    place = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** (low - 1)))).clamp(min=low)
    step = torch.exp2(place - bits)
    return (torch.round(q / step) * step).view(rows, -1)[:, :d], (e + 127).to(torch.uint8)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows, width", [(1, 1), (3, 7), (5, 8), (33, 100), (17, 129), (64, 512), (9, 1001),
                                         (7, 2048), (5, 4099), (3, 8192), (2, 12289), (1, 20000), (1, 65536)])
def test_forward(dtype, rows, width):
    g = gen(rows * width)
    x = rand(g, rows, width, dtype=DT[dtype], shift=0.5)
    res = rand(g, rows, width, dtype=DT[dtype], std=2.0) if width % 2 else None
    w, b = rand(g, width, dtype=DT[dtype], std=0.2, shift=1.0), rand(g, width, dtype=DT[dtype], std=0.3)
    check_forward(x, w, b if rows != 3 else None, res, 1e-5)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("code, group", [("e4m3", 32), ("e4m3", None), ("e5m2", 64), ("e2m1", None)])
@pytest.mark.parametrize("rows, width, want_y", [(40, 33, True), (300, 512, False), (65, 1003, True), (30, 2048, False),
                                                 (11, 8190, False), (3, 16384, True), (2, 30000, False)])
def test_codes(dtype, code, group, rows, width, want_y):
    g = gen(width + rows)
    x = rand(g, rows, width, dtype=DT[dtype])
    x[:, ::17] *= 8
    w, b = rand(g, width, dtype=DT[dtype], std=0.2, shift=1.0), rand(g, width, dtype=DT[dtype], std=0.3)
    res = rand(g, rows, width, dtype=DT[dtype]) if rows % 2 else None
    check_forward(x, w, b, res, 1e-5, code, group, want_y)


def test_codes_where_weight_and_bias_cancel():
    """Outputs near 0 from products and biases that are large: the codes are still those of y."""
    g = gen(5)
    x = rand(g, 64, 512, dtype=torch.float32)
    w = torch.full((512,), 1.0, device="cuda")
    b = -(x[0] - x[0].mean()) / x[0].std(unbiased=False)  # row 0 cancels to rounding
    for code in ("e2m1", "e4m3"):
        r = ops.layer_norm(x[1:], w, b, eps=1e-5, code=code)
        check_forward(x[1:], w, b, None, 1e-5, code)
        assert r.codes is not None


@pytest.mark.parametrize("dtype", list(DT))
def test_means_far_above_the_deviations(dtype):
    g = gen(7)
    x = rand(g, 9, 777, dtype=DT[dtype], std=1.0, shift=900.0)
    w, b = rand(g, 777, dtype=DT[dtype], shift=1.0), rand(g, 777, dtype=DT[dtype])
    check_forward(x, w, b, None, 1e-5, "e4m3")


@pytest.mark.parametrize("scale", [1e-30, 1e30, 3e37])
def test_rows_of_any_magnitude(scale):
    x = rand(gen(8), 5, 300) * scale
    w = torch.ones(300, device="cuda")
    check_forward(x, w, None, None, 0.0)


def test_equal_elements_and_values_that_are_not_finite():
    x = rand(gen(9), 6, 260, dtype=torch.bfloat16)
    x[0] = 3.0
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    x[3] = 0
    w, b = torch.ones(260, dtype=torch.bfloat16, device="cuda"), rand(gen(10), 260, dtype=torch.bfloat16)
    r = ops.layer_norm(x, w, b, code="e2m1")
    assert torch.equal(r.y[0], b) and torch.equal(r.y[3], b)
    assert bool(torch.isnan(r.y[1:3]).all())
    v = ops.unpack4(ops.Codes4(r.codes, r.scales, 260), torch.float32)
    assert bool(torch.isnan(v[1:3]).all()) and bool(torch.isfinite(v[3:]).all())
    check_forward(x[3:], w, b, None, 1e-5, "e2m1")


def test_strides_and_misaligned_views():
    g = gen(11)
    big = rand(g, 40, 1301, dtype=torch.bfloat16)
    x, res = big[3:20, 1:1002], big[20:37, 3:1004]
    w, b = rand(g, 1003, dtype=torch.bfloat16)[1:1002], rand(g, 1002, dtype=torch.bfloat16)[1:]
    check_forward(x, w, b, res, 1e-5, "e4m3", 32)


# ---------------------------------------------------------------- gradient


def check_backward(dy, s, w, ds, weight_dtype=None, **more):
    x = R.f64(s)
    mean = x.mean(1)
    rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + 1e-5)
    mean, rstd = mean.float(), rstd.float()
    want = M.layer_norm_grad(R.f64(dy), x, R.f64(w), mean.double(), rstd.double(),
                             R.f64(ds) if ds is not None else None)
    n, dt = dy.shape[1], dy.dtype
    dx, dw, db = ops.layer_norm_backward(dy, s, w, mean.cuda(), rstd.cuda(), grad_sum=ds,
                                         weight_grad_dtype=weight_dtype, **more)
    # a lane adds up to 64 terms and joins 10 times; ten roundings of a term
    R.close(dx, want[0], want[0].abs() * R.u(dt) * 1.01 + want[3] * 96 * E + R.sub(dt), "dx")
    # a workgroup adds its rows, the parts are joined in 32 slices: under 256 additions here
    wt = weight_dtype or dt
    rows = dy.shape[0]
    adds = 260 if rows < 5000 else 400
    R.close(dw, want[1], want[1].abs() * R.u(wt) * 1.01 + want[4] * adds * E + R.sub(wt), "dw")
    if db is not None:
        R.close(db, want[2], want[2].abs() * R.u(wt) * 1.01 + want[5] * adds * E + R.sub(wt), "db")
    return dx, dw, db


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows, width", [(1, 1), (3, 7), (1, 8), (70, 100), (700, 129), (300, 512), (600, 1001),
                                         (1200, 2048), (50, 4099), (530, 8192), (60, 8193), (300, 12288), (5, 65536)])
def test_backward(dtype, rows, width):
    g = gen(rows + width)
    dt = DT[dtype]
    dy, s = rand(g, rows, width, dtype=dt), rand(g, rows, width, dtype=dt, shift=0.3)
    w = rand(g, width, dtype=dt, std=0.2, shift=1.0)
    ds = rand(g, rows, width, dtype=dt) if width % 2 else None
    check_backward(dy, s, w, ds, torch.float32 if rows % 2 else None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("width", [1, 64, 512, 1001, 8191, 8200])
def test_backward_of_equal_large_elements(dtype, width):
    """mean * rstd passes fp32's range, which nothing of the row itself does."""
    g = gen(width)
    dt = DT[dtype]
    rows = 71
    dy, w = rand(g, rows, width, dtype=dt), rand(g, width, dtype=dt, std=0.2, shift=1.0)
    s = torch.full((rows, width), 2.0 ** 125, dtype=dt, device="cuda")
    s[::2] *= -1
    mean, rstd = s[:, 0].float().contiguous(), torch.full((rows,), 316.0, device="cuda")
    want = M.layer_norm_grad(R.f64(dy), R.f64(s), R.f64(w), R.f64(mean), R.f64(rstd), None)
    dx, dw, db = ops.layer_norm_backward(dy, s, w, mean, rstd)
    # as in check_backward
    R.close(dx, want[0], want[0].abs() * R.u(dt) * 1.01 + want[3] * 96 * E + R.sub(dt), "dx")
    assert not dw.any()
    R.close(db, want[2], want[2].abs() * R.u(dt) * 1.01 + want[5] * 260 * E + R.sub(dt), "db")


def test_backward_without_a_bias_and_into_given_views():
    g = gen(21)
    dt = torch.bfloat16
    dy, s, w = rand(g, 90, 640, dtype=dt), rand(g, 90, 640, dtype=dt), rand(g, 640, dtype=dt, shift=1.0)
    a = check_backward(dy, s, w, None)
    flat = torch.full((3000,), 7.0, dtype=dt, device="cuda")
    x = R.f64(s)
    mean, rstd = x.mean(1), 1 / torch.sqrt(x.var(1, unbiased=False) + 1e-5)
    out, dw, db = ops.layer_norm_backward(dy, s, w, mean.float().cuda(), rstd.float().cuda(), out=dy,
                                          weight_grad_out=flat[101:741], bias_grad_out=flat[741:1381])
    assert out is dy and torch.equal(dy, a[0])
    assert torch.equal(flat[101:741], a[1]) and torch.equal(flat[741:1381], a[2])
    assert bool((flat[:101] == 7).all()) and bool((flat[1381:] == 7).all())
    dy = rand(g, 90, 640, dtype=dt)
    assert ops.layer_norm_backward(dy, s, w, mean.float().cuda(), rstd.float().cuda(), want_bias=False)[2] is None


@pytest.mark.parametrize("width", [640, 10000])
@pytest.mark.parametrize("which", ["dy", "sum", "grad_sum"])
def test_backward_in_place(which, width):
    g = gen(22)
    dt = torch.float16
    t = {"dy": rand(g, 130, width, dtype=dt), "sum": rand(g, 130, width, dtype=dt),
         "grad_sum": rand(g, 130, width, dtype=dt)}
    w = rand(g, width, dtype=dt, shift=1.0)
    mean, rstd = t["sum"].float().mean(1), 1 / t["sum"].float().std(1)
    want = ops.layer_norm_backward(t["dy"], t["sum"], w, mean, rstd, grad_sum=t["grad_sum"])
    got = ops.layer_norm_backward(t["dy"], t["sum"], w, mean, rstd, grad_sum=t["grad_sum"], out=t[which])
    assert got[0] is t[which]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_no_rows():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    f = torch.empty(0, device="cuda")
    assert ops.layer_norm(x, w, code="e2m1").y.shape == (0, 64)
    dx, dw, db = ops.layer_norm_backward(x, x, w, f, f)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    x = torch.empty(0, 9000, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(9000, dtype=torch.bfloat16, device="cuda")
    assert not ops.layer_norm_backward(x, x, w, f, f)[1].any()


def test_strided_gradients():
    g = gen(23)
    big = rand(g, 70, 2100, dtype=torch.bfloat16)
    check_backward(big[:30, 1:1004], big[30:60, 5:1008], rand(g, 1004, dtype=torch.bfloat16)[1:],
                   big[40:70, 1050:2053])


def test_offsets_past_32_bits():
    rows, width = 66000, 65536
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    tail = rand(gen(24), 3, width, dtype=torch.bfloat16)
    x[-3:] = tail
    w, b = rand(gen(25), width, dtype=torch.bfloat16, shift=1.0), rand(gen(26), width, dtype=torch.bfloat16)
    few = ops.layer_norm(tail, w, b, code="e2m1")
    r = ops.layer_norm(x, w, b, code="e2m1")
    assert torch.equal(r.y[-3:], few.y) and torch.equal(r.rstd[-3:], few.rstd)
    assert torch.equal(r.codes.view(torch.uint8)[-3:], few.codes.view(torch.uint8))
    assert torch.equal(r.scales.view(torch.uint8)[:, -3:], few.scales.view(torch.uint8))
    dx, dw, _ = ops.layer_norm_backward(r.y, x, w, r.mean, r.rstd)
    dx3 = ops.layer_norm_backward(few.y, tail, w, few.mean, few.rstd)[0]
    assert torch.equal(dx[-3:], dx3)
    # all the other rows are the same: dy = b, h = 0
    assert bool((dx[1000] == dx[50000]).all())


def test_side_stream_and_graph():
    g = gen(27)
    x, w, b = rand(g, 300, 1000, dtype=torch.bfloat16), rand(g, 1000, dtype=torch.bfloat16), rand(g, 1000, dtype=torch.bfloat16)
    dy = rand(g, 300, 1000, dtype=torch.bfloat16)

    def run():
        r = ops.layer_norm(x, w, b, residual=dy, code="e2m1")
        return (r.y, r.mean, r.codes.view(torch.uint8), r.scales.view(torch.uint8),
                *ops.layer_norm_backward(dy, r.sum, w, r.mean, r.rstd, grad_sum=dy))

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for seed in range(3):
        x.copy_(rand(gen(100 + seed), 300, 1000, dtype=torch.bfloat16))
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, want))


def test_refusals():
    x = rand(gen(28), 4, 64, dtype=torch.bfloat16)
    w = x[0].contiguous()
    f = torch.ones(4, device="cuda")
    for bad in (dict(code="e2m1", group=64), dict(code="e4m3", group=16), dict(code="fp4"),
                dict(bias=w.float()), dict(bias=w[:63]), dict(residual=x.float()), dict(residual=x[:3])):
        with pytest.raises(ValueError):
            ops.layer_norm(x, w, **bad)
    for bad in (dict(weight_grad_dtype=torch.float16), dict(out=x.t()), dict(out=x[:3]), dict(grad_sum=x.half()),
                dict(weight_grad_out=w), dict(weight_grad_out=f[:3]), dict(want_bias=False, bias_grad_out=x[1].clone()),
                dict(weight_grad_out=torch.empty(64, device="cuda"), bias_grad_out=x[1].clone())):
        with pytest.raises(ValueError):
            ops.layer_norm_backward(x, x, w, f, f, **bad)
    both = torch.empty(64, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        ops.layer_norm_backward(x, x, w, f, f, weight_grad_out=both, bias_grad_out=both)
    with pytest.raises(ValueError, match="overlaps"):
        ops.layer_norm_backward(x[1:], x[:3], w, f[:3], f[:3], out=x[:3])
