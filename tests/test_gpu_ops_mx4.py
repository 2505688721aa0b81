"""The 4-bit form and its product against float64: every rounding, both orientations, odd sizes,
strides, values that are not finite, the product's tiles and its form for few tokens, offsets
past 32 bits, side streams and graphs."""
import pytest
import torch

import _more_ref as M
import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops

pytestmark = pytest.mark.gpu
E = R.E
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def rand(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def same(c, x):
    """That a Codes4 is x's (float64), bit for bit."""
    want, byte = M.pack4(x)
    got, gbyte = M.read4(c)
    assert c.width == x.shape[1]
    assert torch.equal(gbyte, byte)
    assert torch.equal(got, want)
    return want, byte


def raw(c):
    return c.codes.view(torch.uint8), c.scales.view(torch.uint8)


# ---------------------------------------------------------------- packing


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows, width", [(1, 1), (1, 32), (2, 33), (5, 100), (128, 128), (129, 127), (300, 513),
                                         (517, 731), (31, 2048), (1030, 40)])
def test_pack(dtype, rows, width):
    g = gen(rows * width)
    x = rand(g, rows, width, dtype=DT[dtype])
    x[:, ::13] *= 20
    x[::7] = 0
    x[rows // 2:] *= 2.0 ** -10
    d = R.f64(x)
    a, b = ops.pack4(x, want="both")
    va, ba = same(a, d)
    vb, bb = same(b, d.t().contiguous())
    for c, one in ((a, ops.pack4(x)), (b, ops.pack4(x, want="columns"))):
        assert all(torch.equal(p, q) for p, q in zip(raw(c), raw(one)))
    for t in DT.values():
        want = M.values4(va, ba, width)
        R.close(ops.unpack4(a, t), want, R.rounded(want, t), "back")
    assert torch.equal(R.f64(ops.unpack4(b, torch.bfloat16)), M.values4(vb, bb, rows))


def test_every_value_of_16_bits():
    """All of bf16's and fp16's values, alone in their group and with each of its neighbours' ends."""
    for dt in (torch.bfloat16, torch.float16):
        v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(dt)
        v = v[torch.isfinite(v.float())]
        x = torch.zeros(v.numel(), 32, dtype=dt)
        x[:, 3] = v
        x[:, 9] = v * 0.25
        x[:, 20] = v * -0.3
        x = x.cuda()
        same(ops.pack4(x), R.f64(x))


def test_ties_and_borders():
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    v = torch.cat([mid, torch.nextafter(mid, torch.zeros(7)), torch.nextafter(mid, torch.full((7,), 9.0))])
    rows = []
    for e in (-140, -126, -120, -60, -1, 0, 1, 60, 120, 125):
        for top in (6.0, 3.01):
            r = torch.zeros(32)
            r[:21], r[21], r[22:29] = v, top, -mid
            rows.append(r.double() * 2.0 ** e)
    x = torch.stack(rows).float().cuda()
    same(ops.pack4(x), R.f64(x))
    six = torch.tensor([6.0, 6.0 + 2.0 ** -21, 6.0 - 2.0 ** -22, 3.0, 1.5]).view(5, 1).cuda()
    same(ops.pack4(six), R.f64(six))
    huge = torch.tensor([[3.4028234e38, 1e38, -2e38, 1e-45]]).cuda()
    same(ops.pack4(huge), R.f64(huge))


def test_groups_that_are_not_finite():
    x = rand(gen(3), 70, 100, dtype=torch.bfloat16)
    x[3, 40], x[9, 99], x[64, 0] = float("nan"), float("inf"), -float("inf")
    a, b = ops.pack4(x, want="both")
    same(a, R.f64(x))
    same(b, R.f64(x).t().contiguous())
    back = ops.unpack4(a, torch.float32)
    assert bool(torch.isnan(back[3, 32:64]).all()) and bool(torch.isnan(back[9, 96:]).all())
    assert bool(torch.isfinite(back[3, :32]).all())


def test_strides_and_misaligned_views():
    big = rand(gen(4), 200, 900, dtype=torch.bfloat16)
    x = big[3:150, 1:700]
    a, b = ops.pack4(x, want="both")
    same(a, R.f64(x))
    same(b, R.f64(x).t().contiguous())
    out = torch.full((200, 900), 5.0, device="cuda", dtype=torch.bfloat16)
    ops.unpack4(a, torch.bfloat16, out=out[1:148, 3:702])
    assert torch.equal(out[1:148, 3:702], ops.unpack4(a, torch.bfloat16))
    out[1:148, 3:702] = 5
    assert bool((out == 5).all())


# ---------------------------------------------------------------- product


def check_product(x, w, dtype, **more):
    a, b = ops.pack4(x), ops.pack4(w)
    xv, wv = R.f64(ops.unpack4(a, torch.float32)), R.f64(ops.unpack4(b, torch.float32))
    got = ops.linear4(a, b, dtype=dtype, **more)
    want, size = xv @ wv.t(), xv.abs() @ wv.abs().t()
    # a rounding for each instruction of 128 and for each join; its own sum is off by one too
    n = x.shape[1] / 128 + 12
    R.close(got, want, want.abs() * R.u(dtype) * 1.01 + size * 2 * n * E + R.sub(dtype), "product")
    return got


SIZES = [(1, 1, 1), (1, 32, 16), (3, 33, 5), (16, 100, 40), (17, 512, 33), (32, 1000, 100), (33, 513, 65), (64, 4096, 96),
         (65, 128, 64), (66, 129, 130), (100, 700, 300), (200, 2048, 257), (300, 1025, 129), (513, 31, 1000),
         (40, 2048, 70), (64, 2300, 200), (65, 2048, 64), (100, 4100, 300), (70, 2561, 65), (200, 22016, 130),
         (33, 1100, 13000)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("tokens, width, features", SIZES)
def test_product(dtype, tokens, width, features):
    g = gen(tokens + width + features)
    x, w = rand(g, tokens, width, dtype=DT[dtype]), rand(g, features, width, dtype=DT[dtype], std=0.1)
    x[:, ::11] *= 10
    got = check_product(x, w, DT[dtype])
    assert torch.equal(ops.linear4(x, ops.pack4(w)), got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tokens, width, features", [(4100, 160, 4300), (1000, 544, 17000), (2304, 96, 8200),
                                                     (2100, 700, 2100), (1030, 1100, 4096), (2048, 300, 2304)])
def test_larger_tiles(tokens, width, features, dtype):
    """256 x 256, also more than one a workgroup, and 128 x 128, whole and ragged."""
    g = gen(tokens)
    x, w = rand(g, tokens, width, dtype=torch.bfloat16), rand(g, features, width, dtype=torch.bfloat16)
    check_product(x, w, dtype)


def test_outputs_that_pass_the_cache():
    """Streamed stores: bit for bit what smaller calls give."""
    g = gen(17)
    x, w = ops.pack4(rand(g, 16400, 96, dtype=torch.bfloat16)), ops.pack4(rand(g, 8300, 96, dtype=torch.bfloat16))
    y = ops.linear4(x, w)
    assert y.numel() * 2 > 256 << 20
    for at in (0, 8192, 16200):
        part = ops.Codes4(x.codes[at:at + 200].contiguous(), x.scales[:, at:at + 200].contiguous(), 96)
        assert torch.equal(y[at:at + 200], ops.linear4(part, w))


@pytest.mark.parametrize("tokens", [5, 40, 100, 1300, 2500])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 7, 8, 9])
def test_every_length_of_the_loop(tokens, steps):
    """k from one step of 128 to nine, and a group short of each."""
    features = {2500: 13000, 1300: 4000}.get(tokens, 200)  # large and middle tiles
    for width in (steps * 128, steps * 128 - 40):
        g = gen(width)
        x, w = rand(g, tokens, width, dtype=torch.bfloat16), rand(g, features, width, dtype=torch.bfloat16)
        a, b = ops.pack4(x), ops.pack4(w)
        xv, wv = ops.unpack4(a, torch.float32).double(), ops.unpack4(b, torch.float32).double()
        got = ops.linear4(a, b, dtype=torch.float32).double()
        size = xv.abs() @ wv.abs().t().contiguous()
        off = (got - xv @ wv.t().contiguous()).abs()
        assert bool((off <= size * 2 * (steps + 12) * E + 1e-38).all())


def test_rows_that_are_not_finite_stay_theirs():
    g = gen(8)
    for tokens in (7, 90):
        x, w = rand(g, tokens, 300), rand(g, 90, 300)
        x[2, 70] = float("nan")
        w[5, 299] = float("inf")
        y = ops.linear4(x, ops.pack4(w))
        bad = torch.zeros(tokens, 90, dtype=torch.bool, device="cuda")
        bad[2], bad[:, 5] = True, True
        assert torch.equal(torch.isnan(y), bad)


def test_scales_far_apart():
    """Products of the largest and least scales: what fp32 holds comes out exactly."""
    x, w = torch.zeros(70, 64, device="cuda"), torch.zeros(70, 64, device="cuda")
    x[:, 0], w[:, 0] = 2.0 ** 120, 2.0 ** -120
    x[:, 40], w[:, 40] = 2.0 ** -100, 3.0 * 2.0 ** 100
    for t in (5, 70):
        assert bool((ops.linear4(x[:t], ops.pack4(w)) == 4.0).all())


def test_strided_outputs_keep_their_neighbours():
    g = gen(9)
    for tokens in (20, 150):
        x, w = rand(g, tokens, 257, dtype=torch.bfloat16), rand(g, 203, 257, dtype=torch.bfloat16)
        for dt in DT.values():
            out = torch.full((tokens + 2, 300), 9.0, dtype=dt, device="cuda")
            view = out[1:tokens + 1, 5:208]
            want = ops.linear4(x, ops.pack4(w), dtype=dt)
            assert ops.linear4(x, ops.pack4(w), out=view) is view
            assert torch.equal(view, want)
            view.fill_(9.0)
            assert bool((out == 9).all())


def test_a_linear_layers_gradients():
    """dx and dw from operands packed along columns, against the products of the values."""
    g = gen(10)
    x, w, dy = rand(g, 150, 210, dtype=torch.bfloat16), rand(g, 90, 210, dtype=torch.bfloat16), rand(g, 150, 90, dtype=torch.bfloat16)
    xr, xc = ops.pack4(x, want="both")
    dr, dc = ops.pack4(dy, want="both")
    dx = ops.linear4(dr, ops.pack4(w, want="columns"), dtype=torch.float32)
    dw = ops.linear4(dc, xc, dtype=torch.float32)

    def v(t):
        a, b = M.pack4(t)
        return M.values4(a, b, t.shape[1])

    for got, p, q in ((dx, v(R.f64(dy)), v(R.f64(w).t().contiguous())),
                      (dw, v(R.f64(dy).t().contiguous()), v(R.f64(x).t().contiguous()))):
        want = p @ q.t()
        R.close(got, want, want.abs() * E + (p.abs() @ q.abs().t()) * 30 * E, "gradient")
    assert xr.width == 210 and xc.width == 150


def test_nothing_to_do():
    w = rand(gen(11), 40, 64, dtype=torch.bfloat16)
    c = ops.pack4(w)
    none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert ops.linear4(none, c).shape == (0, 40)
    assert ops.linear4(w, ops.pack4(none)).shape == (40, 0)
    r, t = ops.pack4(none, want="both")
    assert t.width == 0 and t.codes.shape == (64, 0)
    z = ops.linear4(t, ops.pack4(torch.empty(0, 40, dtype=torch.bfloat16, device="cuda"), want="columns"))
    assert z.shape == (64, 40) and not z.any()
    assert ops.unpack4(r, torch.float32).shape == (0, 64)


def test_offsets_past_32_bits():
    rows, width = 140000, 65536  # codes of 4.6 GB
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    tail = rand(gen(12), 300, width, dtype=torch.bfloat16)
    x[-300:] = tail
    c, few = ops.pack4(x), ops.pack4(tail)
    assert torch.equal(c.codes.view(torch.uint8)[-300:], few.codes.view(torch.uint8))
    assert torch.equal(c.scales.view(torch.uint8)[:, -300:], few.scales.view(torch.uint8))
    back = ops.unpack4(c, torch.bfloat16, out=x)
    assert torch.equal(back[-300:], ops.unpack4(few, torch.bfloat16)) and not back[-600:-300].any()
    for tokens in (9, 130):
        t = ops.pack4(rand(gen(13), tokens, width, dtype=torch.bfloat16))
        y = ops.linear4(t, c)
        # a sum's order is that of k, whatever the tiles
        assert torch.equal(y[:, -300:], ops.linear4(t, few))
        assert not y[:, :-300].any()
    del c, back
    # columns: the transposed codes pass 4 GB as well
    x[:, -3:] = 0
    x[-32:, -1] = 1.0
    k = ops.pack4(x, want="columns")
    codes = k.codes.view(torch.uint8)
    # the least scale with 1 <= 6 * 2^e is 1/4, and 4 is code 6
    assert bool((codes[-1, -16:] == 0x66).all()) and bool((codes[-2:-1, -16:] == 0).all())


def test_two_calls_give_the_same_bits():
    g = gen(14)
    x, w = rand(g, 300, 1000, dtype=torch.bfloat16), ops.pack4(rand(g, 500, 1000, dtype=torch.bfloat16))
    assert torch.equal(ops.linear4(x, w), ops.linear4(x, w))


@pytest.mark.parametrize("tokens", [9, 200])
def test_side_stream_and_graph(tokens):
    g = gen(15)
    x, w = rand(g, tokens, 600, dtype=torch.bfloat16), ops.pack4(rand(g, 700, 600, dtype=torch.bfloat16))

    def run():
        a, b = ops.pack4(x, want="both")
        return (*raw(a), *raw(b), ops.linear4(a, w), ops.linear4(x, w), ops.unpack4(b, torch.float32))

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
        x.copy_(rand(gen(200 + seed), tokens, 600, dtype=torch.bfloat16))
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, want))


def test_refusals():
    x = rand(gen(16), 8, 64, dtype=torch.bfloat16)
    c = ops.pack4(x)
    for call in (lambda: ops.pack4(x, want="cols"), lambda: ops.pack4(x.double()), lambda: ops.pack4(x[0]),
                 lambda: ops.unpack4(c, torch.float64), lambda: ops.unpack4(tuple(c), torch.float32),
                 lambda: ops.unpack4(c._replace(width=65), torch.float32),
                 lambda: ops.unpack4(c._replace(scales=c.scales[:, :7]), torch.float32),
                 lambda: ops.unpack4(c._replace(codes=c.codes[:, :16]), torch.float32),
                 lambda: ops.unpack4(c, torch.float32, out=x), lambda: ops.linear4(x, x),
                 lambda: ops.linear4(x[:, :63], c), lambda: ops.linear4(c, ops.pack4(x[:, :32])),
                 lambda: ops.linear4(c, c, dtype=torch.int32), lambda: ops.linear4(c, c, dtype=torch.float32, out=x[:, :8]),
                 lambda: ops.linear4(c, c, out=x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError, match="overlaps"):
        ops.linear4(c, c, out=c.codes.view(torch.uint8).view(-1).view(torch.bfloat16)[:64].view(8, 8))
