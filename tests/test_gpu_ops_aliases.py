"""Outputs given by the caller that overlap what the call reads: refused, except where the
call allows an input itself, and then right."""
import pytest
import torch

from sharded_optimizer_step_zero_amd import ops

from test_gpu_ops_embed import DEV, gen, rows
from test_gpu_ops_xent import case

pytestmark = pytest.mark.gpu
B = torch.bfloat16


def test_refusals():
    h, w, targets, gloss = case(40, 40, 64, B)
    t, gl = targets.to(DEV), gloss.to(DEV)
    lse = ops.linear_xent(h, w, t)[1]
    ids = torch.zeros(40, dtype=torch.int64, device=DEV)
    big = rows(41, 64, B, 7)
    one, rstd = torch.ones(64, dtype=B, device=DEV), torch.ones(40, device=DEV)
    codes, scales = ops.pack8(h, group=32)
    gates = rows(40, 128, B, 8)
    _, gc, gs = ops.glu(gates, group=32)
    for call in (lambda: ops.linear_xent_backward(h, w, t, lse, gl, weight_grad_out=w),
                 lambda: ops.linear_xent_backward(h, w, t, lse, gl, weight_grad_out=h),
                 lambda: ops.linear_xent_backward(h, w, t, lse, gl, out=w),
                 lambda: ops.linear_xent_backward(big[:40], w, t, lse, gl, out=big[1:]),
                 lambda: ops.linear_xent_backward(h, w, t, lse, gl, out=big[:40], weight_grad_out=big[1:]),
                 lambda: ops.embed(h, ids, out=h), lambda: ops.embed(big[:1], ids, out=big[:40]),
                 lambda: ops.embed_backward(h, ids, 40, out=h),
                 lambda: ops.norm_backward(big[1:], h, one, rstd, out=big[:40]),
                 lambda: ops.norm_backward(h, big[:40], big[40], rstd, out=big[1:]),
                 lambda: ops.norm_backward(h, w, one, rstd, weight_grad_out=one),
                 lambda: ops.norm_backward(big[:40], w, one, rstd, weight_grad_out=big[3]),
                 lambda: ops.unpack8(codes, scales, B, group=32,
                                     out=codes.view(torch.uint8).view(-1)[:40 * 64].view(B).view(20, 64)),
                 lambda: ops.glu_backward(gates[:, :64], gc, gs, group=32, out=gates)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError, match="overlaps"):
        ops.linear_xent_backward(h, w, t, lse, gl, weight_grad_out=w)


@pytest.mark.parametrize("tokens, vocab, width, pad", [(40, 300, 64, 0), (300, 700, 200, 8)])
def test_hidden_itself(tokens, vocab, width, pad):
    h, w, targets, gloss = case(tokens, vocab, width, B, pad)
    t, gl = targets.to(DEV), gloss.to(DEV)
    lse = ops.linear_xent(h, w, t)[1]
    want = ops.linear_xent_backward(h, w, t, lse, gl)
    got = ops.linear_xent_backward(h, w, t, lse, gl, out=h)
    assert got[0] is h and torch.equal(h, want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("n, width", [(700, 40), (33, 520), (3000, 1031), (5, 8192)])
def test_norm_gradient_in_place(n, width):
    one = (1 + 0.1 * torch.randn(width, generator=gen(4))).to(B).to(DEV)
    for which in range(3):
        dy, s, ds = (rows(n, width, B, k) for k in (1, 2, 3))
        rstd = ops.norm(s, one).rstd
        want = ops.norm_backward(dy, s, one, rstd, grad_sum=ds)
        to = (dy, s, ds)[which]
        got = ops.norm_backward(dy, s, one, rstd, grad_sum=ds, out=to)
        assert got[0] is to and torch.equal(to, want[0]) and torch.equal(got[1], want[1])


def test_views_side_by_side():
    """Columns of one buffer do not overlap, whatever lies between their addresses."""
    both = rows(50, 128, B, 1)
    one = torch.ones(64, dtype=B, device=DEV)
    rstd = ops.norm(both[:, :64], one).rstd
    want = ops.norm_backward(rows(50, 64, B, 2), both[:, :64], one, rstd)[0]
    assert torch.equal(ops.norm_backward(rows(50, 64, B, 2), both[:, :64], one, rstd, out=both[:, 64:])[0], want)
