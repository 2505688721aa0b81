"""The softmax statistics of tokens that the model is sure of: a sum of exponentials
that is 1 and little more stays so through every join."""
import pytest
import torch

import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops

from test_gpu_ops_embed import DEV, gen

pytestmark = pytest.mark.gpu


def sure(tokens, vocab, width, dtype, top):
    """Hidden rows of one 1 each, so that logits are entries of w and exact; token t has
    one logit of `top` or more and the rest around 0."""
    h = torch.zeros(tokens, width, dtype=dtype, device=DEV)
    w = torch.randn(vocab, width, generator=gen(1)).to(dtype).to(DEV)
    column = torch.arange(tokens) % width
    h[torch.arange(tokens), column] = 1.0
    targets = (torch.arange(width) * 701 + 13) % vocab
    # values whose product with log2 e is rounded this way and that
    w[targets, torch.arange(width)] = (top * (1 + torch.rand(width, generator=gen(2)) / 4)).to(dtype).to(DEV)
    return h, w, targets[column]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("top", [20.0, 50.0, 100.0, 200.0])
@pytest.mark.parametrize("tokens, vocab", [(64, 50304), (3, 1031), (1000, 20001)])
def test_statistics(dtype, top, tokens, vocab):
    h, w, targets = sure(tokens, vocab, 64, dtype, top)
    loss, lse = ops.linear_xent(h, w, targets.to(DEV))
    want, want_lse = R.xent(h, w, targets)[:2]
    # the sum is 1 and a part in a thousand at most; it is added to 60 times at most (32
    # in a lane, 4 of a tile, 13 of a thread, 8 of a token), half a unit of 1 each, and
    # the logarithm there is as exact; then lse's own rounding
    R.close(lse, want_lse, 64 * R.E + want_lse.abs() * R.E, "lse")
    R.close(loss, want, 64 * R.E + want * 2 * R.E, "loss")
    assert (loss >= 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens, vocab", [(64, 50304), (1000, 20001)])
def test_gradient_pulls_the_target_up(dtype, tokens, vocab):
    """p - 1 is never positive."""
    for top in (9.0, 20.0, 50.0, 100.0):
        h, w, targets = sure(tokens, vocab, 64, dtype, top)
        t = targets.to(DEV)
        lse = ops.linear_xent(h, w, t)[1]
        dw = ops.linear_xent_backward(h, w, t, lse, torch.ones(tokens, device=DEV), want_hidden=False)[1]
        first = targets[:64].to(DEV)[:min(tokens, 64)]
        assert (dw[first, torch.arange(first.numel(), device=DEV)] <= 0).all(), top
