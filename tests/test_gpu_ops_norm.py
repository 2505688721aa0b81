"""The norm with residual and 8-bit output, 8-bit activations and the gated unit on
the GPU against float64."""
import pytest
import torch

import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops

from test_gpu_ops_embed import DEV, TYPES, gen, rows

pytestmark = pytest.mark.gpu
NARROW = [torch.bfloat16, torch.float16]


# ------------------------------------------------------------------ norm

NORM = [  # rows, width, pad, off
    (1, 1, 0, 0), (3, 7, 0, 0), (5, 8, 0, 0), (33, 64, 0, 0), (9, 100, 0, 0), (17, 128, 4, 0),
    (4, 512, 8, 8), (5, 520, 0, 0), (3, 1024, 0, 1), (2, 1031, 0, 0), (3, 2048, 0, 0), (2, 4096, 0, 0),
    (2, 4104, 0, 0), (2, 8192, 0, 0), (1, 16384, 0, 0), (1, 20001, 0, 0), (1, 65536, 0, 0), (1300, 72, 0, 0)]
# fp32 roundings of rstd: each lane adds 64 squares at most, 10 steps join a
# workgroup's lanes and waves (16 waves in a chain); half of it through the root,
# and the mean, eps, root and quotient
RSTD = 0.5 * (64 + 1 + 6 + 16) + 5


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n, width, pad, off", NORM)
def test_norm(dtype, n, width, pad, off):
    x, r = rows(n, width, dtype, 1, pad, off), rows(n, width, dtype, 2, pad, off)
    w = (1 + 0.1 * torch.randn(width, generator=gen(3))).to(dtype).to(DEV)
    for residual, code, group, want_y in ((r, "e4m3", 128, True), (None, "e5m2", 32, True), (r, "e4m3", 64, False),
                                          (None, None, 128, True), (r, "e5m2", 64, True)):
        out = ops.norm(x, w, residual=residual, eps=1e-5, code=code, group=group, want_y=want_y)
        if residual is None:
            assert out.sum is x
        else:
            total = R.f64(x) + R.f64(r)
            R.close(out.sum, total, R.rounded(total, dtype, 1), "sum")
        y, rstd = R.norm(R.f64(out.sum), R.f64(w), 1e-5)
        R.close(out.rstd, rstd, rstd * RSTD * R.E, "rstd")
        assert (out.y is not None) == want_y
        if want_y:
            R.close(out.y, y, R.rounded(y, dtype, RSTD + 2), "y")
        if code is None:
            assert out.codes is None and out.scales is None
            continue
        byte = R.byte_of(out.scales)
        assert byte.shape == (n, -(-width // group)) and out.codes.dtype == R.CODE_DTYPE[code]
        d = (RSTD + 2) * R.E
        scale = torch.exp2(byte.double() - 127).repeat_interleave(group, 1)[:, :width]
        R.close(R.unpack(out.codes, byte, group), y,
                y.abs() * (R.CODE_U[code] + 2 * d) + scale * R.CODE_SUB[code], "codes")
        # the scale is the least power of two that holds the group, up to y's own error
        full = torch.zeros(n, byte.shape[1] * group, dtype=torch.float64)
        full[:, :width] = y.abs()
        amax = full.view(n, -1, group).amax(2)
        top = 1.75 * torch.exp2(byte.double() - 127 + R.TOP[code])
        assert (amax <= top * (1 + d)).all() and ((amax >= top / 2 * (1 - d)) | (byte == 0)).all()


def test_norm_in_place_and_rows_apart():
    """sum may be the residual itself; a row that is not finite spoils only itself."""
    x, r = rows(4, 256, torch.bfloat16, 1), rows(4, 256, torch.bfloat16, 2)
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    out = ops.norm(x, w, residual=r, code="e4m3", group=64)
    y = out.y.float().cpu()
    assert torch.isfinite(y[[0, 3]]).all() and torch.isnan(y[1]).all() and torch.isnan(y[2, 200])
    byte = R.byte_of(out.scales)
    assert (byte[1] == 255).all() and byte[2, 3] == 255 and (byte[[0, 3]] < 255).all()
    # an infinite sum of squares: rstd is 0, the other groups are zeros
    assert (byte[2, :3] == 0).all() and not out.codes[2, :192].float().any()
    s = r.clone()
    ops.zs_norm_forward(x.data_ptr(), 256, s.data_ptr(), 256, w.data_ptr(), s.data_ptr(), 256, None, 256, None, None,
                        out.rstd.data_ptr(), 4, 256, 1e-6, ops.ZS_BF16, 0, 128,
                        torch.cuda.current_stream().cuda_stream)
    assert torch.equal(s.view(torch.int16), out.sum.view(torch.int16))
    # a row of zeros
    z = ops.norm(torch.zeros_like(x), w, eps=1e-6, code="e4m3")
    assert not z.y.any() and (R.byte_of(z.scales) == 0).all() and torch.isfinite(z.rstd).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n, width, pad, off", NORM + [(0, 64, 0, 0), (0, 600, 0, 0), (700, 1040, 0, 0)])
def test_norm_backward(dtype, n, width, pad, off):
    s, dy, ds = (rows(n, width, dtype, k, pad, off) for k in (1, 2, 3))
    w = (1 + 0.1 * torch.randn(width, generator=gen(4))).to(dtype).to(DEV)
    rstd = ops.norm(s, w, eps=1e-5).rstd if n else torch.empty(0, device=DEV)
    for grad_sum in (None, ds):
        dx, dw = ops.norm_backward(dy, s, w, rstd, grad_sum=grad_sum, weight_grad_dtype=torch.float32)
        wx, ww, sx, sw = R.norm_grad(R.f64(dy), R.f64(s), R.f64(w), R.f64(rstd),
                                     None if grad_sum is None else R.f64(ds))
        # the row's dot product: 64 a lane, joined as rstd's; then a handful of products
        R.close(dx, wx, sx * (64 + 1 + 6 + 16 + 10) * R.E + R.rounded(wx, dtype), "dx")
        R.close(dw, ww, sw * (n + 2 + 32) * R.E + 1e-45, "dw")
        assert torch.equal(dx, ops.norm_backward(dy, s, w, rstd, grad_sum=grad_sum)[0])
    dx2, dw2 = ops.norm_backward(dy, s, w, rstd, grad_sum=ds, out=dy)  # in place
    assert dx2 is dy and torch.equal(dx2, dx)
    assert torch.equal(dw2, dw.to(dtype))


# ------------------------------------------------------------------ 8 bits


def specials(dtype):
    """Rows whose groups hold zeros, one subnormal, the type's extremes, exact borders of
    the scale, infinities and NaN."""
    x = torch.randn(12, 200, generator=gen(5))
    x[0] = 0
    x[1] *= torch.finfo(dtype).smallest_normal / 16
    x[2, 3] = torch.finfo(dtype).max
    x[3, :] = 1.75
    x[4, :] = 1.7578125
    x[5, 0], x[5, 130] = float("inf"), float("-inf")
    x[6, 50] = float("nan")
    x[7] *= 1e-3
    x[7, 64] = 1000.0
    x[8] = torch.linspace(-448, 448, 200)
    x[9] = -0.0
    x[10, 199] = 60000.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("code", ["e4m3", "e5m2"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_pack_is_exact(dtype, code, group):
    """The scaling is exact and the rounding is one: codes and scales bit for bit."""
    cases = [specials(dtype).to(DEV)] + [rows(n, d, dtype, 6, pad, off) for n, d, pad, off in (
        (1, 1, 0, 0), (3, 31, 0, 0), (5, 129, 3, 0), (7, 1000, 0, 0), (2, 2048, 8, 8), (3, 4100, 0, 1), (0, 40, 0, 0),
        (300, 136, 0, 0))]
    for x in cases:
        codes, scales = ops.pack8(x, code=code, group=group)
        want, byte = R.pack(x, code, group)
        assert torch.equal(R.byte_of(scales), byte)
        same = codes.cpu().view(torch.uint8) == want.view(torch.uint8)
        # a zero's sign follows the input's
        assert same.all(), (x.shape, int((~same).sum()))
        for dt in TYPES:
            back = ops.unpack8(codes, scales, dt, group=group)
            value = R.unpack(want, byte, group)
            expect = value.float().to(dt)
            assert torch.equal(torch.isnan(back).cpu(), torch.isnan(value))
            fine = ~torch.isnan(value)
            assert torch.equal(back.cpu()[fine], expect[fine])
        to = rows(x.shape[0], x.shape[1], dtype, 7, 8, 0)
        ops.unpack8(codes, scales, dtype, group=group, out=to)
        assert torch.equal(torch.nan_to_num(to), torch.nan_to_num(ops.unpack8(codes, scales, dtype, group=group)))


GLU = [(1, 1, 0, 0), (3, 8, 0, 0), (5, 33, 0, 0), (4, 128, 0, 0), (3, 1000, 8, 8), (2, 2736, 0, 0), (3, 5000, 0, 1),
       (0, 64, 0, 0), (600, 40, 4, 0), (2, 11008, 0, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("n, width, pad, off", GLU)
def test_glu(dtype, act, n, width, pad, off):
    x = rows(n, 2 * width, dtype, 8, pad, off)
    if n > 2:
        x[1] *= 30  # far out on both sides
    g, u = R.f64(x[:, :width]), R.f64(x[:, width:])
    a, _, e, _ = R.act(g, act)
    tiny = 2.0 ** -100 * (1 + u.abs())  # past fp32's exponential the sigmoid is 0
    for code, group in (("e4m3", 128), ("e5m2", 32)):
        out, codes, scales = ops.glu(x, act=act, code=code, group=group)
        R.close(out, a * u, (a * u).abs() * e * R.E + R.rounded(a * u, dtype, 2) + tiny, "out")
        for half in (0, 1):
            want, byte = R.pack(x[:, half * width:(half + 1) * width], code, group)
            assert torch.equal(R.byte_of(scales)[:, half], byte)
            assert torch.equal(codes.cpu().view(torch.uint8)[:, half * width:(half + 1) * width],
                               want.view(torch.uint8))
        dout = rows(n, width, dtype, 9, pad, off)
        byte = R.byte_of(scales)
        cg, cu = (R.unpack(codes[:, h * width:(h + 1) * width], byte[:, h], group) for h in (0, 1))
        f, slope, e8, size = R.act(cg, act)
        do = R.f64(dout)
        dgu, again = ops.glu_backward(dout, codes, scales, act=act, group=group, want_out=True)
        tiny8 = 2.0 ** -100 * (1 + cu.abs()) * (1 + do.abs())
        R.close(dgu[:, :width], do * cu * slope,
                (do * cu).abs() * size * (3 * e8 + 8) * R.E + R.rounded(do * cu * slope, dtype, 2) + tiny8, "dgate")
        R.close(dgu[:, width:], do * f, (do * f).abs() * e8 * R.E + R.rounded(do * f, dtype, 2) + tiny8, "dup")
        R.close(again, f * cu, (f * cu).abs() * e8 * R.E + R.rounded(f * cu, dtype, 2) + tiny8, "out again")
        to = rows(n, 2 * width, dtype, 10, pad, off)
        assert ops.glu_backward(dout, codes, scales, act=act, group=group, out=to)[1] is None
        assert torch.equal(to, dgu)
    out2, none, none2 = ops.glu(x, act=act, code=None)
    assert none is None and none2 is None and torch.equal(out2, out)


def test_glu_of_values_that_are_not_finite():
    x = torch.ones(2, 256, dtype=torch.bfloat16, device=DEV)
    x[0, 3], x[0, 128 + 70] = float("nan"), float("inf")
    for act in ("silu", "gelu"):
        out, codes, scales = ops.glu(x, act=act, group=32)
        assert torch.isnan(out[0, 3]) and torch.isinf(out[0, 70]) and int((~torch.isfinite(out)).sum()) == 2
        assert (R.byte_of(scales) == 255).nonzero().tolist() == [[0, 0, 0], [0, 1, 2]]
        dgu, _ = ops.glu_backward(torch.ones(2, 128, dtype=torch.bfloat16, device=DEV), codes, scales, act=act, group=32)
        bad = torch.zeros(2, 256, dtype=torch.bool)
        bad[0, :32] = bad[0, 128:160] = bad[0, 64:96] = True  # d(gate) there takes the infinite up
        assert torch.equal(torch.isnan(dgu).cpu(), bad)
    # the largest inputs of the type
    x = torch.full((1, 256), 3e38, dtype=torch.bfloat16, device=DEV)
    x[0, :64] = -3e38
    for act in ("silu", "gelu"):
        _, codes, scales = ops.glu(x, act=act, group=32)
        dgu, _ = ops.glu_backward(torch.full((1, 128), 1e-38, dtype=torch.bfloat16, device=DEV), codes, scales, act=act,
                                  group=32)
        assert torch.isfinite(dgu).all()


def test_norm_and_act8_refuse():
    x, w = rows(4, 64, torch.bfloat16, 1), torch.ones(64, dtype=torch.bfloat16, device=DEV)
    rstd = torch.ones(4, device=DEV)
    codes, scales = ops.pack8(x, group=32)
    gl = ops.glu(x, group=32)
    for call in (lambda: ops.norm(x.t(), w), lambda: ops.norm(x, w.float()), lambda: ops.norm(x, w[:32]),
                 lambda: ops.norm(x, w, residual=x[:3]), lambda: ops.norm(x, w, residual=x.half()),
                 lambda: ops.norm(x, w, code="int8"), lambda: ops.norm(x, w, code="e4m3", group=100),
                 lambda: ops.norm(x, w[::2]), lambda: ops.norm(x.int(), w),
                 lambda: ops.norm_backward(x, x, w, rstd[:3]), lambda: ops.norm_backward(x, x.half(), w, rstd),
                 lambda: ops.norm_backward(x, x, w, rstd.double()), lambda: ops.norm_backward(x, x, w, rstd, grad_sum=x[:2]),
                 lambda: ops.norm_backward(x, x, w, rstd, weight_grad_dtype=torch.float16),
                 lambda: ops.pack8(x, code="e3m4"), lambda: ops.pack8(x, group=16), lambda: ops.pack8(x[:, ::2]),
                 lambda: ops.unpack8(codes, scales, torch.int32, group=32),
                 lambda: ops.unpack8(codes, scales, torch.float32, group=64),
                 lambda: ops.unpack8(codes, scales.view(torch.uint8), torch.float32, group=32),
                 lambda: ops.unpack8(codes.view(torch.uint8), scales, torch.float32, group=32),
                 lambda: ops.unpack8(codes[:, :32], scales, torch.float32, group=32),
                 lambda: ops.glu(x[:, :63]), lambda: ops.glu(x, act="relu"), lambda: ops.glu(x, group=256),
                 lambda: ops.glu_backward(x, gl[1], gl[2], group=32),
                 lambda: ops.glu_backward(x[:, :48], *ops.glu(rows(4, 96, torch.bfloat16, 1), group=32)[1:], group=64),
                 lambda: ops.glu_backward(x[:, :32], gl[1], gl[2], act="tanh", group=32),
                 lambda: ops.glu_backward(x[:3, :32], gl[1], gl[2], group=32)):
        with pytest.raises(ValueError):
            call()
