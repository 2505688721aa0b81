"""The hinge next to its border: the forward and the backward pass take the same side of it."""
import pytest
import torch

from sharded_optimizer_step_zero_amd import ops

pytestmark = pytest.mark.gpu

# m - 1; all of these margins are exact in fp64, and those within 2^-25 below 1 are 1 to the nearest in fp32
OFF = [-0.5, -2.0 ** -24, -3 * 2.0 ** -26, -2.0 ** -25, -2.0 ** -26, -2.0 ** -30, -2.0 ** -50, 0.0, 2.0 ** -50,
       2.0 ** -30, 2.0 ** -24, 2.0 ** -23, 0.5]


@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("off", OFF)
def test_a_hinge_that_costs_has_a_gradient(off, average):
    # m = (sum of the rejected) - (sum of the chosen) = 1 + off, each of two sequences of one token
    chosen = max(0.0, -off)
    rejected = 1.0 + max(0.0, off)
    if rejected != torch.tensor(rejected, dtype=torch.float32).item():  # a token's loss has 24 bits
        chosen, rejected = -off, 1.0
    loss = torch.tensor([chosen, rejected], device="cuda")
    o = torch.tensor([0, 1, 2], device="cuda")
    kw = dict(beta=1.0, kind="hinge", average=average)
    r = ops.preference_loss(loss, None, o, **kw)
    d = ops.preference_loss_backward(r, o, torch.full((1,), 0.5, device="cuda"), 2, **kw)
    assert float(r.loss) == max(0.0, -off)
    # within a step of fp32 (2^-24 below 1, 2^-23 above)
    assert abs(float(r.margins) - (1.0 + off)) <= 2.0 ** -24
    assert d.tolist() == ([0.5, -0.5] if off < 0 else [0.0, 0.0])


@pytest.mark.parametrize("kind", ["sigmoid", "squared"])
def test_the_other_kinds_margins_are_the_nearest(kind):
    loss = torch.tensor([2.0 ** -30, 1.0], device="cuda")
    r = ops.preference_loss(loss, None, torch.tensor([0, 1, 2], device="cuda"), beta=1.0, kind=kind)
    assert float(r.margins) == 1.0
