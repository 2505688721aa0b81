"""The cross entropy's products as training sizes run them: large tiles with many steps and a
ragged end of k, several pieces of the vocabulary, and the small tiles beside them.  Which
case takes which path is checked without a GPU, in test_ops_xent_plan.py."""
import pytest
import torch

import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops

from test_gpu_ops_embed import DEV, gen, rows

pytestmark = pytest.mark.gpu

CASES = {  # (tokens, vocab, width): what the plan has to be
    # 256 x 256 tiles of all three products; k of 33 steps, the last of 8 and of 52
    (2100, 8300, 2056): dict(small=0, small_h=0, small_w=0, pieces=1, last=8300, splits=3, copy_w=0),
    # the same of copied rows, and vocabulary entries past the last whole chunk
    (2100, 8301, 2050): dict(small=0, small_h=0, small_w=0, pieces=1, last=8301, splits=3, copy_w=1),
    # two pieces, the last one shorter and ragged
    (8200, 17003, 2056): dict(small=0, small_h=0, small_w=0, pieces=2, last=8299, splits=1, copy_w=0),
    # two pieces, small tiles for grad_weight, whose width is less than one of them
    (8200, 17003, 72): dict(small=0, small_h=0, small_w=1, pieces=2, last=8299, splits=7, copy_w=0),
    # few tokens: small tiles of the logits, every workgroup beginning at a step of its own
    (100, 9001, 2056): dict(small=1, small_h=1, small_w=0, pieces=1, last=9001, splits=7, copy_w=0),
    (40, 2000, 2040): dict(small=1, small_h=1, small_w=1, pieces=1, last=2000, splits=4, copy_w=0),
}


def whole(n, d, dtype, seed, scale):
    """Small whole numbers times a power of two, so that logits are exact in fp32."""
    return (torch.randint(-2, 3, (n, d), generator=gen(seed)).double() * scale).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens, vocab, width", CASES)
def test_products(dtype, tokens, vocab, width):
    h, w = whole(tokens, width, dtype, 1, 1.0), whole(vocab, width, dtype, 2, 2.0 ** -5 if width > 500 else 2.0 ** -2)
    targets = torch.randint(0, vocab, (tokens,), generator=gen(3)).to(DEV)
    targets[::7] = -100
    targets[3::50] = vocab
    targets[1], targets[2] = 0, vocab - 1
    gloss = (torch.rand(tokens, generator=gen(4)) + 0.5).to(DEV)
    # float64, on the GPU
    hd, wd = h.double(), w.double()
    live = (targets >= 0) & (targets < vocab)
    at = targets.clamp(0, vocab - 1)[:, None]
    g = torch.mm(hd, wd.t().contiguous())
    lse = torch.logsumexp(g, 1)
    span = float((g.amax(1) - g.amin(1)).max())
    want = torch.where(live, lse - g.gather(1, at)[:, 0], torch.zeros_like(lse))
    got, got_lse = ops.linear_xent(h, w, targets)
    # the logits are exact: sums of exponentials (60 terms in a row), and an exponential whose
    # argument is rounded twice; the logarithm and the last sum
    e = (64 + 4 * min(span, 60)) * R.E
    R.close(got_lse, lse.cpu(), e + 4 * lse.abs().cpu() * R.E, "lse")
    R.close(got, want.cpu(), 2 * e + 8 * lse.abs().cpu() * R.E, "loss")
    g = torch.exp(g - lse[:, None])
    # p - 1 at the target cancels: its error is relative to p + 1
    size = g.scatter_add(1, at, torch.ones_like(lse)[:, None])
    g.scatter_add_(1, at, -torch.ones_like(lse)[:, None])
    weight = torch.where(live, gloss.double(), torch.zeros_like(lse))[:, None]
    g *= weight
    # G's half step of its type, p's error, and fp16's least subnormal below the largest of G
    least = 2.0 ** -15 * R.sub(torch.float16) * 1.5 if dtype == torch.float16 else 0.0
    off = g.abs() * R.u(dtype) + size * weight * (2 * e + 8 * float(lse.abs().max()) * R.E) + least * (weight > 0)
    size = g.abs() + off
    dh, dw = ops.linear_xent_backward(h, w, targets, got_lse, gloss)
    for out, ref, err, n in ((dh, torch.mm(g, wd), torch.mm(off, wd.abs()) + torch.mm(size, wd.abs()) * vocab * R.E, 0),
                             (dw, torch.mm(g.t().contiguous(), hd), torch.mm(off.t().contiguous(), hd.abs())
                              + torch.mm(size.t().contiguous(), hd.abs()) * tokens * R.E, 1)):
        R.close(out, ref.cpu(), err.cpu() + R.rounded(ref.cpu(), dtype, 4), "gradient of " + ("hidden", "weight")[n])
    # into strided destinations, one at a time: the same bits
    to = rows(tokens, width, dtype, 9, 5, 1)
    ops.linear_xent_backward(h, w, targets, got_lse, gloss, out=to, want_weight=False)
    assert torch.equal(to, dh)
    to = rows(vocab, width, dtype, 9, 8, 8)
    ops.linear_xent_backward(h, w, targets, got_lse, gloss, weight_grad_out=to, want_hidden=False)
    assert torch.equal(to, dw)
