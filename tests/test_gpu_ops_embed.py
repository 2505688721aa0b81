"""The embedding and its gradient on the GPU against float64."""
import pytest
import torch

import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(n, d, dtype, seed, pad=0, off=0):
    """[n, d] on the GPU; with pad or off, a view with a longer row stride that starts
    off elements into its storage."""
    x = torch.randn(n, d, generator=gen(seed)).to(dtype)
    big = torch.full((n * (d + pad) + off + 8,), 7.0, dtype=dtype, device=DEV)
    v = big[off:off + n * (d + pad)].view(n, d + pad)[:, :d]
    v.copy_(x)
    return v


FORWARD = [  # tokens, vocab, width, pad, off
    (1, 1, 1, 0, 0), (3, 5, 8, 0, 0), (32, 1000, 2048, 0, 0), (7, 50, 63, 0, 0), (9, 50, 64, 3, 0),
    (9, 50, 72, 8, 8), (5, 11, 4104, 0, 1), (257, 33, 520, 0, 0), (2, 3, 8200, 0, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens, vocab, width, pad, off", FORWARD)
def test_embed(dtype, tokens, vocab, width, pad, off):
    table = rows(vocab, width, dtype, 1, pad, off)
    for ids_dtype, start in ((torch.int64, 0), (torch.int32, 5)):
        ids = torch.randint(-3, vocab + 3, (tokens,), generator=gen(2)).to(ids_dtype) + start
        want = R.embed(table, ids, 1.5, start)
        out = ops.embed(table, ids.to(DEV), scale=1.5, vocab_start=start)
        R.close(out, want, R.rounded(want, dtype, 1), "embed")
        to = rows(tokens, width, dtype, 3, pad, off)
        assert ops.embed(table, ids.to(DEV), scale=1.5, vocab_start=start, out=to) is to
        assert torch.equal(to, out)


def test_embed_shapes_and_nothing():
    table = rows(10, 16, torch.bfloat16, 1)
    ids = torch.randint(0, 10, (2, 3), generator=gen(1)).to(DEV)
    out = ops.embed(table, ids)
    assert out.shape == (2, 3, 16) and torch.equal(out, table[ids])
    assert ops.embed(table, ids[:0]).shape == (0, 3, 16)
    assert ops.embed_backward(out, ids, 10).shape == (10, 16)
    # no tokens: a gradient of zeros, and nothing to add
    g = ops.embed_backward(out[:0], ids[:0], 10)
    assert g.shape == (10, 16) and not g.any()
    g.fill_(3)
    ops.embed_backward(out[:0], ids[:0], 10, out=g, accumulate=True)
    assert (g == 3).all()


BACKWARD = [  # tokens, vocab, width, what ids, pad, off
    (1, 1, 1, "random", 0, 0), (1, 7, 8, "random", 0, 0), (31, 5, 16, "random", 0, 0),
    (32, 5, 16, "same", 0, 0), (33, 5, 16, "same", 0, 0), (64, 3, 40, "same", 0, 0),
    (1000, 17, 63, "random", 0, 0), (1000, 17, 64, "random", 5, 0), (1000, 2000, 72, "random", 8, 8),
    (4097, 300, 520, "skewed", 0, 0), (4097, 300, 520, "skewed", 0, 1), (3000, 140_000, 24, "skewed", 0, 0),
    (3000, 9, 1032, "none", 0, 0), (2049, 600_001, 8, "random", 0, 0), (70_000, 512, 8, "skewed", 0, 0),
    (2000, 1_000, 8, "bucket", 0, 0)]


def make_ids(kind, tokens, vocab, seed):
    g = gen(seed)
    if kind == "same":
        return torch.full((tokens,), vocab - 1)
    if kind == "none":
        return torch.full((tokens,), -100)
    if kind == "bucket":  # all ids of one bucket of the sort
        return torch.randint(0, vocab // 256 + 1, (tokens,), generator=g) * 256 % vocab
    if kind == "skewed":
        return ((vocab + 1.0) ** torch.rand(tokens, generator=g)).long().clamp(0, vocab) - 1
    return torch.randint(-2, vocab + 2, (tokens,), generator=g)


def grad_bound(dtype, want, size, count):
    """fp32 sums of `count` terms, the scale's product and one rounding."""
    return size * (count + 2) * R.E + R.rounded(want, dtype, 2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens, vocab, width, kind, pad, off", BACKWARD)
def test_embed_backward(dtype, tokens, vocab, width, kind, pad, off):
    ids = make_ids(kind, tokens, vocab, 4)
    dout = rows(tokens, width, dtype, 5, pad, off)
    want, size, count = R.embed_grad(dout, ids, vocab, 0.75)
    got = ops.embed_backward(dout, ids.to(DEV), vocab, scale=0.75)
    R.close(got, want, grad_bound(dtype, want, size, count), "gradient")
    again = ops.embed_backward(dout, ids.to(DEV), vocab, scale=0.75)
    assert torch.equal(got, again)
    # fp32 output, shifted int32 ids, a strided destination
    to = rows(vocab, width, torch.float32, 6, pad, off)
    ops.embed_backward(dout, (ids + 9).int().to(DEV), vocab, scale=0.75, vocab_start=9, out=to)
    R.close(to, want, grad_bound(torch.float32, want, size, count), "fp32 gradient")
    # added to what is there; rows without tokens keep their bits
    base = rows(vocab, width, dtype, 7)
    to = base.clone()
    ops.embed_backward(dout, ids.to(DEV), vocab, scale=0.75, out=to, accumulate=True)
    total = R.f64(base) + want
    R.close(to, total, grad_bound(dtype, total, size + R.f64(base).abs(), count + 1), "added gradient")
    bare = (count[:, 0] == 0).to(DEV)
    assert torch.equal(to[bare], base[bare])


def test_embed_backward_keeps_nan_of_skipped_tokens_out():
    ids = torch.tensor([1, -100, 2, 1, 5])
    dout = torch.ones(5, 24, dtype=torch.bfloat16, device=DEV)
    dout[1] = float("nan")
    dout[4] = float("inf")
    g = ops.embed_backward(dout, ids.to(DEV), 4)
    assert torch.equal(g[:, 0].cpu().float(), torch.tensor([0.0, 2.0, 1.0, 0.0]))
    dout[2] = float("nan")
    g = ops.embed_backward(dout, ids.to(DEV), 4).cpu()
    assert torch.isnan(g[2]).all() and torch.isfinite(g[[0, 1, 3]]).all()


def test_embed_offsets_past_32_bits():
    """A table of more than 2^32 bytes and 2^31 elements."""
    vocab, width = 540_000, 4096
    table = torch.zeros(vocab, width, dtype=torch.bfloat16, device=DEV)
    table[-1] = 3.0
    table[524_288 - 1] = 2.0
    ids = torch.tensor([vocab - 1, 524_287, 0], device=DEV)
    out = ops.embed(table, ids)
    assert (out[0] == 3).all() and (out[1] == 2).all() and (out[2] == 0).all()
    g = table
    ops.embed_backward(out, ids, vocab, out=g)
    assert (g[-1] == 3).all() and (g[524_287] == 2).all() and int((g != 0).any(1).sum()) == 2


def test_embed_refuses():
    t, i = rows(10, 16, torch.bfloat16, 1), torch.zeros(4, dtype=torch.int64, device=DEV)
    d = rows(4, 16, torch.bfloat16, 1)
    for call in (lambda: ops.embed(t.t(), i), lambda: ops.embed(t[:, ::2], i), lambda: ops.embed(t, i.float()),
                 lambda: ops.embed(t, i.cpu()), lambda: ops.embed(t, i[::2]), lambda: ops.embed(t[0], i),
                 lambda: ops.embed(t.long(), i), lambda: ops.embed(t, i, out=d[:3]),
                 lambda: ops.embed(t, i, out=d.float()), lambda: ops.embed(t[:1].expand(10, 16), i),
                 lambda: ops.embed_backward(d[:3], i, 10), lambda: ops.embed_backward(d, i, 0),
                 lambda: ops.embed_backward(d, i, 10, accumulate=True),
                 lambda: ops.embed_backward(d, i, 10, out=t.half()),
                 lambda: ops.embed_backward(d, i, 10, out_dtype=torch.float16),
                 lambda: ops.embed_backward(d, i, 10, out=t[:, :8]),
                 lambda: ops.embed_backward(d, i, 10, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            call()
