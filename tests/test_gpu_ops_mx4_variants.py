"""The kernels of the 4-bit form that only some sizes reach: packing both ways or along columns by
the large blocks, their own conversions on every 16-bit value, ties and borders, and the
product of few tokens with many features."""
import pytest
import torch

import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops
from test_gpu_ops_mx4 import DT, check_product, gen, rand, raw, same

pytestmark = pytest.mark.gpu
LARGE = 1024  # blocks of 256 x 256 from which on packing takes them


def blocks(rows, width, both):
    """Of 256 x 256, whole spans of 512 along what is packed."""
    return -(-rows // 512) * 2 * (-(-width // 512) * 2 if both else -(-width // 256))


def same_bits(a, b):
    assert a.width == b.width
    for p, q in zip(raw(a), raw(b)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows, width", [(5133, 13307), (13307, 5133), (262145, 33)])
def test_large_blocks(dtype, rows, width):
    """Bit for bit what the kernel along rows gives of the matrix and of its transpose, which other
    tests compare with float64."""
    for both in (True, False):
        assert blocks(rows, width, both) >= LARGE
    x = rand(gen(rows), rows, width, dtype=DT[dtype])
    x[:, ::13] *= 20
    x[::7] = 0
    x[rows // 2:] *= 2.0 ** -10
    x[5, 3], x[rows - 1, width - 1], x[rows // 3, width // 2] = float("nan"), float("inf"), -float("inf")
    a, b = ops.pack4(x, want="both")
    along = ops.pack4(x)
    same_bits(a, along)
    del a, along
    columns = ops.pack4(x.t().contiguous())
    same_bits(b, columns)
    del b
    same_bits(ops.pack4(x, want="columns"), columns)


def both_ways(x):
    """That every way of packing x, whose values are x's in float64, gives its form."""
    d, t = R.f64(x), x.t().contiguous()
    a, other = ops.pack4(x, want="both")
    same(a, d)
    _, b = ops.pack4(t, want="both")
    same_bits(b, a)
    same_bits(ops.pack4(t, want="columns"), a)
    same_bits(ops.pack4(x, want="columns"), other)
    same_bits(ops.pack4(x), a)
    # the same rows often enough for large blocks
    rows = x.shape[0]
    n = -(-LARGE * 256 // rows)
    many = x.repeat(n, 1)
    turned = many.t().contiguous()
    assert min(blocks(*many.shape, True), blocks(*turned.shape, True), blocks(*turned.shape, False)) >= LARGE
    codes, scales = raw(a)
    for c in (ops.pack4(many, want="both")[0], ops.pack4(turned, want="both")[1], ops.pack4(turned, want="columns")):
        p, q = raw(c)
        assert torch.equal(p.view(n, *codes.shape), codes.expand(n, *codes.shape))
        q = q.view(q.shape[0], n, rows, 4, 4)
        assert torch.equal(q, scales[:, None].expand_as(q))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_value_of_16_bits(dtype):
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(DT[dtype])
    v = v[torch.isfinite(v.float())]
    x = torch.zeros(v.numel(), 32, dtype=DT[dtype])
    x[:, 3] = v
    x[:, 9] = v * 0.25
    x[:, 20] = v * -0.3
    both_ways(x.cuda())


@pytest.mark.parametrize("dtype", list(DT))
def test_ties_and_borders(dtype):
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    near = [mid * (1 + s * torch.finfo(DT[dtype]).eps) for s in (-1, 1)]
    rows = []
    for e in (-140, -126, -120, -60, -20, -14, -1, 0, 1, 8, 60, 120, 125):
        for top in (6.0, 3.0, 3.0 * (1 + torch.finfo(DT[dtype]).eps)):
            r = torch.zeros(32)
            r[:7], r[7:14], r[14:21], r[21], r[22:29] = mid, *near, top, -mid
            rows.append(r.double() * 2.0 ** e)
    x = torch.stack(rows).float().to(DT[dtype])
    both_ways(x[torch.isfinite(x.float()).all(1)].cuda())


FEW = [(1, 520, 8161), (16, 1000, 8200), (9, 4100, 9001), (17, 96, 8161), (29, 1100, 8200), (32, 4096, 8192), (31, 700, 20011)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("tokens, width, features", FEW)
def test_few_tokens_and_many_features(dtype, tokens, width, features):
    """32 features a workgroup, for one and for two sixteens of tokens."""
    assert -(-features // 32) >= 256 and tokens <= 32
    g = gen(tokens + features)
    x, w = rand(g, tokens, width, dtype=DT[dtype]), rand(g, features, width, dtype=DT[dtype], std=0.1)
    x[:, ::11] *= 10
    got = check_product(x, w, DT[dtype])
    assert torch.equal(ops.linear4(x, ops.pack4(w)), got)


def test_few_tokens_keep_the_neighbours_of_a_strided_output():
    x, w = rand(gen(1), 27, 300, dtype=torch.bfloat16), ops.pack4(rand(gen(2), 8203, 300, dtype=torch.bfloat16))
    out = torch.full((30, 8300), 9.0, dtype=torch.bfloat16, device="cuda")
    want = ops.linear4(x, w)
    ops.linear4(x, w, out=out[1:28, 5:8208])
    assert torch.equal(out[1:28, 5:8208], want)
    out[1:28, 5:8208] = 9.0
    assert bool((out == 9).all())


def test_the_largest_magnitudes_read_back_as_infinity():
    """From 3.5 * 2^126 on the nearest code is 4 of the scale 2^126: 2^128, which no type here holds."""
    below, at, top = 3.5 * 2.0 ** 126 * (1 - 2.0 ** -24), 3.5 * 2.0 ** 126, torch.finfo(torch.float32).max
    x = torch.zeros(3, 32)
    x[0, 0], x[1, 0], x[2, 0] = below, at, -top
    x = x.cuda()
    for c in (ops.pack4(x), ops.pack4(x, want="both")[0], ops.pack4(x.t().contiguous(), want="columns")):
        same(c, R.f64(x))
        for dt in (torch.float32, torch.bfloat16):
            v = ops.unpack4(c, dt)
            assert v[:, 0].tolist() == [3 * 2.0 ** 126, float("inf"), -float("inf")]
            assert not v[:, 1:].any()


@pytest.mark.parametrize("tokens, features", [(5, 70), (70, 70), (3000, 4400)])
def test_the_product_takes_the_largest_and_the_least_values_as_they_are(tokens, features):
    x, w = torch.zeros(tokens, 64, device="cuda"), torch.zeros(features, 64, device="cuda")
    x[:, 0], x[:, 40] = 3.4e38, -3.4e38  # 2^128 in the 4-bit form
    w[:, 0], w[:, 40] = 2.0 ** -100, 2.0 ** -101
    assert bool((ops.linear4(x, ops.pack4(w), dtype=torch.float32) == 2.0 ** 27).all())
    x.zero_()
    w.zero_()
    x[:, 0], x[:, 3], w[:, 0] = 2.0 ** -128, 2.0 ** -127, 2.0 ** 100  # a scale of 2^-127
    assert bool((ops.linear4(x, ops.pack4(w), dtype=torch.float32) == 2.0 ** -28).all())
