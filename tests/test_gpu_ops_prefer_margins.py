"""The preference loss and its gradient where a pair's margin is infinite: the chosen or the
rejected sequence has a token that the policy or the reference gives no probability.  The formulas
have values there, which are told by hand."""
import math

import pytest
import torch

import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops

pytestmark = pytest.mark.gpu
INF = float("inf")
KINDS = [("sigmoid", 0.0), ("sigmoid", 0.25), ("hinge", 0.0), ("squared", 0.0)]

# the margin's sign by where the infinity stands: a = -sum(loss - ref), m = beta (a_chosen - a_rejected)
PLACES = [("loss", 0, -INF), ("loss", 1, INF), ("ref", 0, INF), ("ref", 1, -INF)]


def at_infinity(m, kind, smoothing):
    """(loss, slope) of a pair whose margin is +-infinity"""
    if kind == "sigmoid":  # -(1 - s) log sigma(m) - s log sigma(-m), the second term absent without s
        loss = INF if m < 0 or smoothing else 0.0
        return loss, -(1.0 - smoothing) if m < 0 else smoothing
    if kind == "hinge":
        return (INF, -1.0) if m < 0 else (0.0, 0.0)
    return INF, m


def run(loss, ref, o, grad, **kw):
    r = ops.preference_loss(loss, ref, o, **kw)
    return r, ops.preference_loss_backward(r, o, grad, loss.numel(), **kw)


@pytest.mark.parametrize("kind, smoothing", KINDS)
@pytest.mark.parametrize("place", PLACES, ids=["loss-chosen", "loss-rejected", "ref-chosen", "ref-rejected"])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("tokens", [60, 200000])  # a workgroup for a pair, and sequences divided over workgroups
def test_a_token_without_probability(kind, smoothing, place, average, tokens):
    which, seq, m = place
    g = torch.Generator(device="cuda").manual_seed(tokens)
    loss = torch.rand(tokens, generator=g, device="cuda") + 0.5
    ref = loss + torch.randn(tokens, generator=g, device="cuda") * 0.1
    o = [0, tokens // 4, tokens // 2, tokens // 2 + 7, tokens - 5]
    offsets = torch.tensor(o, device="cuda")
    assert (ops.zs_prefer_workspace_bytes(tokens, 2) > 256) == (tokens > 60)
    mask = torch.ones(tokens, dtype=torch.bool, device="cuda")
    mask[1::9] = False
    grad = torch.tensor([0.75, -0.5], device="cuda")
    kw = dict(beta=0.5, kind=kind, smoothing=smoothing, average=average, mask=mask)
    plain, plain_d = run(loss, ref, offsets, grad, **kw)
    at = o[seq] + 3
    assert bool(mask[at])
    (loss if which == "loss" else ref)[at] = INF
    got, d = run(loss, ref, offsets, grad, **kw)

    want, slope = at_infinity(m, kind, smoothing)
    assert float(got.margins[0]) == m and float(got.loss[0]) == want
    a = INF if (which == "ref") else -INF
    assert float(got.rewards[0, seq]) == a and math.isfinite(float(got.rewards[0, 1 - seq]))
    counted = mask.cpu()
    for i in (0, 1):
        n = int(counted[o[i]:o[i + 1]].sum())
        each = slope * 0.5 * 0.75 / (n if average else 1) * (1 if i else -1)
        part = d[o[i]:o[i + 1]].cpu().double()
        inside = counted[o[i]:o[i + 1]]
        expect = torch.where(inside, torch.full_like(part, each), torch.zeros_like(part))
        # the factor is taken in fp64 and rounded once
        bound = 0.0 if math.isinf(each) else R.rounded(expect, torch.float32)
        R.close(part, expect, bound, "gradient")
    # the other pair's values and what lies in no sequence stay as they are
    for x, y in zip(got, plain):
        assert torch.equal(x[1], y[1])
    assert torch.equal(d[o[2]:], plain_d[o[2]:])


@pytest.mark.parametrize("kind, smoothing", KINDS)
def test_both_sides_without_probability_have_no_margin(kind, smoothing):
    loss = torch.tensor([INF, INF, 1.0, 2.0], device="cuda")
    o = torch.arange(5, device="cuda")
    got, d = run(loss, None, o, torch.ones(2, device="cuda"), kind=kind, smoothing=smoothing)
    assert bool(torch.isnan(got.loss[0])) and bool(torch.isnan(d[:2]).all())
    assert bool(torch.isfinite(got.loss[1])) and bool(torch.isfinite(d[2:]).all())
