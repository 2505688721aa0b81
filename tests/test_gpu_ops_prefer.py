"""The preference loss and its gradient against float64: kinds, masks, empty sequences, padding
behind the last one, sequences divided over workgroups, offsets that are wrong, side streams
and graphs."""
import pytest
import torch

import _more_ref as M
import _ops_ref as R
from sharded_optimizer_step_zero_amd import ZeroShardError, ops

pytestmark = pytest.mark.gpu
E = R.E
KINDS = [("sigmoid", 0.0), ("sigmoid", 0.1), ("hinge", 0.0), ("squared", 0.0)]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def case(tokens, pairs, seed, tail=3, head=2):
    g = gen(seed)
    loss = -torch.log(torch.rand(tokens, generator=g, device="cuda").clamp(min=1e-6))
    ref = loss + torch.randn(tokens, generator=g, device="cuda") * 0.1
    cut = torch.randint(head, max(head + 1, tokens - tail), (2 * pairs - 1,), generator=g, device="cuda").sort().values
    o = torch.cat([torch.tensor([head], device="cuda"), cut, torch.tensor([max(head, tokens - tail)], device="cuda")])
    mask = torch.rand(tokens, generator=g, device="cuda") < 0.8
    grad = torch.rand(pairs, generator=g, device="cuda") - 0.2
    return loss, ref, o, mask, grad


def check(loss, ref, o, mask, grad, beta, kind, margin=0.0, smoothing=0.0, average=False):
    kw = dict(beta=beta, kind=kind, smoothing=smoothing, average=average, mask=mask)
    r = ops.preference_loss(loss, ref, o, margin=margin, **kw)
    d = ops.preference_loss_backward(r, o, grad, loss.numel(), **kw)
    # masked places hold anything
    l2 = loss if mask is None else torch.where(mask, loss, torch.zeros_like(loss))
    r2 = ref if mask is None or ref is None else torch.where(mask, ref, torch.zeros_like(ref))
    want, rewards, m, lengths, size, slope, g = M.prefer(l2, r2, o, mask, beta, kind, margin, smoothing, average, grad)
    b32 = float(torch.tensor(beta, dtype=torch.float32))
    tiny = size * 2.0 ** -40
    # beta, margin and smoothing reach the kernel in fp32
    R.close(r.rewards, rewards * (b32 / beta), R.rounded(rewards, torch.float32, 1) + tiny, "rewards")
    mbound = (rewards.abs().sum(1) + abs(margin)) * 1.5 * E + tiny.sum(1)
    R.close(r.margins, m, R.rounded(m, torch.float32) + mbound, "margins")
    assert torch.equal(r.lengths.cpu().long(), lengths)
    lbound = slope.abs() * mbound + abs(smoothing) * E * (m.abs() + 1) + mbound ** 2 / beta ** 2
    R.close(r.loss, want, R.rounded(want, torch.float32, 4) + lbound + 1e-12, "loss")
    # the margin is rounded once more before its slope is taken
    if kind == "hinge":
        near = (m - 1).abs() <= m.abs() * E + mbound
        assert not bool(near.any())
    moved = {"sigmoid": 0.25, "hinge": 0.0, "squared": 2 / beta ** 2}[kind]
    sb = slope.abs() * 6 * E + moved * (m.abs() * E + mbound) + smoothing * E
    scale = torch.zeros(loss.numel()).double()
    for i in range(len(o) - 1):
        n = max(1, int(lengths.view(-1)[i])) if average else 1
        scale[int(o[i]):int(o[i + 1])] = float(sb[i // 2] * R.f64(grad)[i // 2].abs()) * beta / n
    R.close(d, g, scale * 1.01 + g.abs() * 2 * E + 1e-38, "gradient")
    return r, d


@pytest.mark.parametrize("kind, smoothing", KINDS)
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("tokens, pairs", [(2, 1), (30, 1), (700, 4), (5000, 33), (3000, 700)])
def test_losses_and_gradients(kind, smoothing, average, tokens, pairs):
    loss, ref, o, mask, grad = case(tokens, pairs, tokens + pairs)
    for r, m in ((ref, mask), (None, mask), (ref, None)):
        check(loss, r, o, m, grad, 0.3, kind, 0.25 if kind != "squared" else 0.0, smoothing, average)
    check(loss, ref, o.int(), mask, grad, 1.0, kind, 0.0, smoothing, average)


@pytest.mark.parametrize("pairs", [1, 3, 100])
def test_long_sequences_are_divided(pairs):
    tokens = 1 << 21
    assert ops.zs_prefer_workspace_bytes(tokens, pairs) > 256
    loss, ref, o, mask, grad = case(tokens, pairs, 5)
    check(loss, ref, o, mask, grad, 0.1, "sigmoid")
    check(loss, None, o, mask, grad, 2.0, "sigmoid", average=True)


def test_masked_places_hold_anything():
    loss, ref, o, mask, grad = case(900, 5, 6)
    want = [t.clone() for t in (*ops.preference_loss(loss, ref, o, mask=mask),)]
    loss[~mask], ref[~mask] = float("nan"), float("inf")
    r, d = check(loss, ref, o, mask, grad, 0.1, "sigmoid")
    assert all(torch.equal(a, b) for a, b in zip(r, want))
    assert bool((d[~mask] == 0).all()) and bool(torch.isfinite(d).all())
    # and outside the sequences
    loss[:2], loss[-3:] = float("nan"), float("nan")
    assert all(torch.equal(a, b) for a, b in zip(ops.preference_loss(loss, ref, o, mask=mask), want))


@pytest.mark.parametrize("kind, smoothing", KINDS)
def test_empty_sequences_and_masks_that_leave_nothing(kind, smoothing):
    loss, ref, _, _, _ = case(40, 1, 7)
    o = torch.tensor([0, 0, 0, 10, 10, 25, 40], device="cuda")
    mask = torch.ones(40, dtype=torch.bool, device="cuda")
    mask[10:25] = False
    grad = torch.ones(3, device="cuda")
    for average in (False, True):
        r, d = check(loss, ref, o, mask, grad, 0.5, kind, 0.0, smoothing, average)
        assert r.rewards[0].tolist() == [0, 0] and r.lengths.tolist() == [[0, 0], [10, 0], [0, 15]]
        assert not d[10:25].any()
        mask8 = mask.to(torch.uint8) * 3  # any byte that is not 0 counts
        assert torch.equal(ops.preference_loss(loss, ref, o, beta=0.5, kind=kind, smoothing=smoothing,
                                               average=average, mask=mask8).loss, r.loss)


@pytest.mark.parametrize("empty", [1, 2, 3, 3001])
def test_many_empty_sequences_between_two_tokens(empty):
    """A thread's four tokens on either side of them, at each place among the four."""
    for at in (4, 5, 6, 7):
        o = torch.tensor([0, 3] + [at] * (empty + 1) + [9, 17][:2 - empty % 2], device="cuda")
        pairs = (len(o) - 1) // 2
        g = gen(at)
        loss = torch.rand(20, generator=g, device="cuda")
        grad = torch.rand(pairs, generator=g, device="cuda") + 0.1
        check(loss, None, o, None, grad, 0.5, "sigmoid")


def test_no_tokens_and_no_pairs():
    none = torch.empty(0, device="cuda")
    o = torch.zeros(5, dtype=torch.int64, device="cuda")
    r = ops.preference_loss(none, None, o)
    R.close(r.loss, torch.full((2,), 0.6931471805599453).double(), E, "loss")
    assert ops.preference_loss_backward(r, o, torch.ones(2, device="cuda"), 0).shape == (0,)
    o = o[:1]
    r = ops.preference_loss(torch.ones(9, device="cuda"), None, o)
    assert r.loss.shape == (0,) and r.rewards.shape == (0, 2)
    assert not ops.preference_loss_backward(r, o, none, 9).any()


@pytest.mark.parametrize("m", [-200.0, -30.0, 0.0, 30.0, 200.0, 1e4])
def test_margins_far_out(m):
    """The sigmoid's loss and slope where one side has no digits left in 1 - sigma."""
    loss = torch.tensor([0.0, m], device="cuda")
    o = torch.tensor([0, 1, 2], device="cuda")
    check(loss, None, o, None, torch.ones(1, device="cuda"), 1.0, "sigmoid")
    check(loss, None, o, None, torch.ones(1, device="cuda"), 1.0, "sigmoid", smoothing=0.25)


def test_values_that_are_not_finite_go_through():
    loss = torch.tensor([1.0, float("nan"), 2.0, 3.0], device="cuda")
    o = torch.arange(5, device="cuda")
    for kind in ("sigmoid", "hinge", "squared"):
        r = ops.preference_loss(loss, None, o, kind=kind)
        d = ops.preference_loss_backward(r, o, torch.ones(2, device="cuda"), 4, kind=kind)
        assert bool(torch.isnan(r.loss[0])) and bool(torch.isfinite(r.loss[1]))
        assert bool(torch.isnan(d[:2]).all()) and bool(torch.isfinite(d[2:]).all())


def test_wrong_offsets_stay_in_bounds():
    loss = torch.ones(100, device="cuda")
    for o in ([-5, 20, 300], [50, 10, 90], [200, 300, 400], [-(1 << 40), 1 << 40, 1 << 50], [90, 40, 10]):
        o = torch.tensor(o, device="cuda")
        r = ops.preference_loss(loss, None, o)
        assert bool(torch.isfinite(r.loss).all())
        d = ops.preference_loss_backward(r, o, torch.ones(1, device="cuda"), 100)
        assert bool(torch.isfinite(d).all())


def test_side_stream_and_graph():
    loss, ref, o, mask, grad = case(100000, 4, 9)
    assert ops.zs_prefer_workspace_bytes(100000, 4) > 256

    def run():
        r = ops.preference_loss(loss, ref, o, mask=mask)
        return (*r, ops.preference_loss_backward(r, o, grad, loss.numel(), mask=mask))

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
        new = case(100000, 4, 20 + seed)
        for to, t in zip((loss, ref, o, mask, grad), new):
            to.copy_(t)
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, want))


def test_refusals():
    loss, ref, o, mask, grad = case(100, 2, 10)
    r = ops.preference_loss(loss, ref, o)
    for call in (lambda: ops.preference_loss(loss.half(), ref, o), lambda: ops.preference_loss(loss, ref[:99], o),
                 lambda: ops.preference_loss(loss, ref, o[:4]), lambda: ops.preference_loss(loss, ref, o.float()),
                 lambda: ops.preference_loss(loss, ref, o, kind="ipo"), lambda: ops.preference_loss(loss, ref, o, mask=mask[:99]),
                 lambda: ops.preference_loss(loss, ref, o, mask=mask.float()),
                 lambda: ops.preference_loss(loss.view(10, 10), ref, o), lambda: ops.preference_loss(loss, ref, o.cpu()),
                 lambda: ops.preference_loss_backward(r, o, grad[:1], 100),
                 lambda: ops.preference_loss_backward(r, o[:3], grad, 100),
                 lambda: ops.preference_loss_backward(r, o, grad, 100, out=torch.empty(99, device="cuda")),
                 lambda: ops.preference_loss_backward(r._replace(lengths=r.lengths.long()), o, grad, 100)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ZeroShardError, match="beta"):
        ops.preference_loss(loss, ref, o, beta=0.0)
    with pytest.raises(ValueError, match="overlaps"):
        ops.preference_loss_backward(r, o, grad, 2, out=grad)
