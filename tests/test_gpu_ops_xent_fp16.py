"""Gradients of the cross entropy in fp16: G's entries far below the largest keep
their digits, as the type's fifteen binades above 1 allow."""
import pytest
import torch

import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops

from test_gpu_ops_embed import DEV, gen, rows

pytestmark = pytest.mark.gpu
TOP = 2.0 ** 15  # G's largest magnitude in fp16


def gradients(h, w, targets, gloss):
    """Both gradients against float64.  G is off by half a step of fp16 and, where it is
    subnormal, by half the least subnormal under TOP; then fp32 sums and the last rounding."""
    t = targets.to(DEV)
    loss, lse, logits, err, g, dh, dw, live, hh, ww = R.xent(h, w, targets, gloss)
    got_lse = ops.linear_xent(h, w, t)[1]
    got = ops.linear_xent_backward(h, w, t, got_lse, gloss.to(DEV))
    at = targets.clamp(0, w.shape[0] - 1)[:, None]
    p = torch.exp(logits - lse[:, None])
    # p - 1 at the target cancels: its error is relative to p + 1
    size = g.abs() + torch.zeros_like(g).scatter_(1, at, (gloss.double() * 2 * p.gather(1, at)[:, 0])[:, None])
    # the logits' own error, lse's (a chain of a hundred sums at most) and an exponential
    # whose argument, within 60, is rounded twice
    e = 2 * float(err.max()) + (100 + 120 + 4 * float(lse.abs().max())) * R.E
    sub = torch.full_like(g, float(gloss.max()) * R.sub(torch.float16) / TOP)
    for out, want, by in ((got[0], dh, lambda x: x @ ww.abs()), (got[1], dw, lambda x: x.t().contiguous() @ hh.abs())):
        length = g.shape[1] if out is got[0] else g.shape[0]
        bound = by(size) * (R.u(torch.float16) + e + (length + 8) * 2 * R.E) + by(sub)
        R.close(out, want, bound + R.rounded(want, torch.float16, 4), "gradient")


@pytest.mark.parametrize("tokens, vocab, width", [(60, 3001, 64), (600, 6000, 128)])
def test_improbable_entries(tokens, vocab, width):
    """A head that has learned frequencies: most of the vocabulary lies many binades
    below the targets, and rows without a target have nothing else."""
    h = rows(tokens, width, torch.float16, 1)
    w = rows(vocab, width, torch.float16, 2) * (2.0 / width ** 0.5)
    h[:, 0] = 1.0
    w[:, 0] = -14.0 * torch.rand(vocab, generator=gen(3)).to(DEV)
    targets = torch.randint(0, vocab // 3, (tokens,), generator=gen(4))
    gradients(h, w, targets, torch.full((tokens,), 8.0))


def test_tokens_of_little_weight():
    """Weights over a factor of 10^6: the light tokens' rows keep their digits."""
    tokens, vocab, width = 130, 500, 64
    h, w = rows(tokens, width, torch.float16, 1), rows(vocab, width, torch.float16, 2) * 0.25
    targets = torch.randint(0, vocab, (tokens,), generator=gen(4))
    gloss = 4096.0 * 10.0 ** (-6 * torch.rand(tokens, generator=gen(5)))
    gradients(h, w, targets, gloss)


@pytest.mark.parametrize("power", [-140, -100, -60, 60, 100, 126])
def test_any_size_of_the_loss_gradient(power):
    """The factor that G carries comes back whole at either end of fp32: results past fp16
    are zeros and infinities, and no NaN."""
    h, w = rows(40, 64, torch.float16, 1), rows(300, 64, torch.float16, 2) * 0.25
    t = torch.randint(0, 300, (40,), generator=gen(4)).to(DEV)
    gl = (torch.rand(40, generator=gen(5)) + 0.5).to(DEV)
    lse = ops.linear_xent(h, w, t)[1]
    one = ops.linear_xent_backward(h, w, t, lse, gl)
    other = ops.linear_xent_backward(h, w, t, lse, gl * 2.0 ** power)
    for a, b in zip(one, other):
        assert torch.equal(b, (a.double() * 2.0 ** power).half())
