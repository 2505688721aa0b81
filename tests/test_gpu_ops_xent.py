"""The cross entropy of a linear head and its gradient on the GPU against float64,
and the operators on side streams and in graphs."""
import pytest
import torch

import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops

from test_gpu_ops_embed import DEV, gen, rows

pytestmark = pytest.mark.gpu
HALVES = [torch.bfloat16, torch.float16]

SHAPES = [  # tokens, vocab, width, pad, off, one multi-piece case last
    (1, 1, 1, 0, 0), (1, 1000, 64, 0, 0), (2, 7, 9, 0, 0), (63, 129, 72, 0, 0), (64, 256, 128, 8, 8),
    (65, 257, 100, 0, 0), (128, 300, 64, 3, 0), (129, 515, 136, 0, 0), (256, 512, 64, 0, 0), (257, 1000, 200, 0, 1),
    (300, 70, 264, 0, 0), (5, 5000, 1032, 0, 0), (700, 777, 30, 0, 0), (8200, 8300, 40, 0, 0)]


def case(tokens, vocab, width, dtype, pad=0, off=0, seed=1):
    h, w = rows(tokens, width, dtype, seed, pad, off), rows(vocab, width, dtype, seed + 1, pad, off)
    w.mul_(2.0 / width ** 0.5)
    targets = torch.randint(0, vocab, (tokens,), generator=gen(seed + 2))
    skip = torch.rand(tokens, generator=gen(seed + 3)) < 0.1
    targets[skip] = torch.where(torch.rand(int(skip.sum()), generator=gen(seed + 4)) < 0.5, -100, vocab)
    gloss = torch.rand(tokens, generator=gen(seed + 5)) + 0.5
    return h, w, targets, gloss


def loss_bound(logits, err, lse):
    """The logits' error, the sum of exponentials (a chain of 32 or so terms in a
    lane, the tile's, then up to 64 parts and 16 threads) and an exponential whose
    argument is rounded, the logarithm and the last sum."""
    span = (logits.amax(1) - logits.amin(1)).clamp(max=60)
    return err.amax(1) + (160 + 4 * span) * R.E + (lse.abs() + 2) * 4 * R.E


def check_grad(dtype, got, want, size, err, length):
    """size: the sum of |G| times |the other factor|; err: a bound of the logits' and
    lse's errors, which G has relative; the half-step of rounding G, fp32 sums of
    `length` products, and the last rounding."""
    R.close(got, want, size * (R.u(dtype) + 3 * err + (length + 8) * 2 * R.E) + R.rounded(want, dtype, 4), "gradient")


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("tokens, vocab, width, pad, off", SHAPES)
def test_linear_xent(dtype, tokens, vocab, width, pad, off):
    h, w, targets, gloss = case(tokens, vocab, width, dtype, pad, off)
    loss, lse, logits, err, g, dh, dw, live, hh, ww = R.xent(h, w, targets, gloss)
    bound = loss_bound(logits, err, lse)
    for td in (torch.int64, torch.int32):
        t = targets.to(td).to(DEV)
        got, got_lse = ops.linear_xent(h, w, t)
        R.close(got_lse, lse, bound, "lse")
        R.close(got, loss, 2 * bound, "loss")
        assert not got[~live.to(DEV)].any()
    gl = gloss.to(DEV)
    got_dh, got_dw = ops.linear_xent_backward(h, w, t, got_lse, gl)
    # p - 1 at the target cancels: its error is relative to p + 1
    at = targets.clamp(0, vocab - 1)[:, None]
    p = torch.exp(logits - lse[:, None])
    gsize = g.abs() + torch.zeros_like(g).scatter_(1, at, torch.where(live, gloss.double() * 2 * p.gather(1, at)[:, 0],
                                                                    torch.zeros(()).double())[:, None])
    # fp16 holds small entries of G, divided by the largest gradient, to half its least subnormal
    gsize = gsize + torch.where(live, 1.0, 0.0).double()[:, None] * float(gloss.max()) * R.sub(dtype) / R.u(dtype)
    e = float((err.amax(1) + bound).max()) + 70 * R.E
    check_grad(dtype, got_dh, dh, gsize @ ww.abs(), e, vocab)
    check_grad(dtype, got_dw, dw, gsize.t().contiguous() @ hh.abs(), e, tokens)
    # one at a time, into strided destinations, twice the same bits
    to = rows(tokens, width, dtype, 9, pad, off)
    a, b = ops.linear_xent_backward(h, w, t, got_lse, gl, out=to, want_weight=False)
    assert a is to and b is None and torch.equal(to, got_dh)
    to = rows(vocab, width, dtype, 9, pad, off)
    a, b = ops.linear_xent_backward(h, w, t, got_lse, gl, weight_grad_out=to, want_hidden=False)
    assert a is None and b is to and torch.equal(to, got_dw)


@pytest.mark.parametrize("dtype", HALVES)
def test_no_token_counts(dtype):
    """Nothing but padding, whose hidden rows and gradients are not even finite."""
    h, w, _, _ = case(70, 300, 64, dtype)
    h.fill_(float("nan"))
    t = torch.full((70,), -100, device=DEV)
    gl = torch.full((70,), float("inf"), device=DEV)
    loss, lse = ops.linear_xent(h, w, t)
    assert not loss.any()
    dh, dw = ops.linear_xent_backward(h, w, t, lse, gl)
    assert not dh.any() and not dw.any()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("tokens", [40, 300])
def test_values_that_are_not_finite_stay_in_their_rows(dtype, tokens):
    h, w, targets, gloss = case(tokens, 300, 64, dtype)
    targets[:4] = torch.tensor([5, -100, 7, 9])
    clean = ops.linear_xent(h, w, targets.to(DEV))
    gl = gloss.to(DEV)
    clean_dh, clean_dw = ops.linear_xent_backward(h, w, targets.to(DEV), clean[1], gl)
    h[1] = float("nan")  # padding
    gl[1] = float("nan")
    h[2, 3] = float("inf")
    loss, lse = ops.linear_xent(h, w, targets.to(DEV))
    keep = torch.arange(tokens, device=DEV) != 2
    assert torch.equal(loss[keep], clean[0][keep]) and not torch.isfinite(loss[2])
    dh, dw = ops.linear_xent_backward(h, w, targets.to(DEV), lse, gl)
    assert torch.equal(dh[keep], clean_dh[keep]) and not torch.isfinite(dh[2]).all()
    assert not torch.isfinite(dw).all()
    h[2, 3] = 0.5
    targets[2] = -100
    lse = ops.linear_xent(h, w, targets.to(DEV))[1]
    assert torch.isfinite(ops.linear_xent_backward(h, w, targets.to(DEV), lse, gl)[1]).all()


def test_large_logits():
    """Logits in the thousands: the maximum comes out before the exponential."""
    h = torch.zeros(3, 8, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(600, 8, dtype=torch.bfloat16, device=DEV)
    h[:, 0] = torch.tensor([1.0, -1.0, 0.0])
    w[:, 0] = torch.linspace(-4096, 4096, 600)
    t = torch.tensor([599, 599, 0], device=DEV)
    loss, lse = ops.linear_xent(h, w, t)
    want = R.xent(h, w, t)
    R.close(lse, want[1], 4096 * 8 * R.E + 100 * R.E, "lse")
    R.close(loss, want[0], 4096 * 16 * R.E + 100 * R.E, "loss")
    dh, dw = ops.linear_xent_backward(h, w, t, lse, torch.ones(3, device=DEV))
    assert torch.isfinite(dh).all() and torch.isfinite(dw).all()


def test_no_tokens():
    w = rows(300, 64, torch.bfloat16, 1)
    h, t, f = w[:0], torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV)
    loss, lse = ops.linear_xent(h, w, t)
    assert loss.shape == lse.shape == (0,)
    dh, dw = ops.linear_xent_backward(h, w, t, f, f)
    assert dh.shape == (0, 64) and dw.shape == (300, 64) and not dw.any()


def test_small_gradients_keep_their_digits():
    """grad_loss far below the 16-bit types' range comes back in the last rounding only."""
    h, w, targets, gloss = case(200, 400, 64, torch.bfloat16)
    t = targets.to(DEV)
    lse = ops.linear_xent(h, w, t)[1]
    one = ops.linear_xent_backward(h, w, t, lse, gloss.to(DEV))
    small = ops.linear_xent_backward(h, w, t, lse, gloss.to(DEV) * 2.0 ** -60)
    for a, b in zip(one, small):
        assert torch.equal(a, (b.double() * 2.0 ** 60).to(a.dtype))


def everything(s):
    """One pass through every operator; returns all outputs."""
    x = ops.embed(s["table"], s["ids"], scale=2.0)
    n = ops.norm(x, s["w"], residual=s["r"], code="e4m3", group=64)
    out, codes, scales = ops.glu(n.y, group=32)
    loss, lse = ops.linear_xent(out, s["head"], s["targets"])
    dh, dhead = ops.linear_xent_backward(out, s["head"], s["targets"], lse, s["gl"])
    dgu, again = ops.glu_backward(dh, codes, scales, group=32, want_out=True)
    dx, dw = ops.norm_backward(dgu, n.sum, s["w"], n.rstd, grad_sum=s["r"])
    back = ops.unpack8(n.codes, n.scales, torch.bfloat16, group=64)
    c2, s2 = ops.pack8(dx, code="e5m2")
    dt = ops.embed_backward(dx, s["ids"], 500, scale=2.0)
    return [x, n.y, n.sum, n.rstd, n.codes, n.scales, out, codes, scales, loss, lse, dh, dhead, dgu, again, dx, dw,
            back, c2, s2, dt]


def state(seed, tokens=300):
    b = torch.bfloat16
    return dict(table=rows(500, 512, b, seed), ids=torch.randint(-1, 500, (tokens,), generator=gen(seed)).to(DEV),
                w=rows(1, 512, b, seed + 1)[0].contiguous(), r=rows(tokens, 512, b, seed + 2),
                head=rows(700, 256, b, seed + 3), targets=torch.randint(-1, 700, (tokens,), generator=gen(seed)).to(DEV),
                gl=torch.rand(tokens, generator=gen(seed + 4)).to(DEV))


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


def test_side_stream():
    s = state(1)
    want = everything(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        late = {k: torch.empty_like(v) for k, v in s.items()}
        torch.cuda._sleep(50_000_000)  # the inputs arrive late on this stream
        for k in s:
            late[k].copy_(s[k])
        got = everything(late)
    side.synchronize()
    assert same(got, want)


def test_graph():
    """A captured pass replayed on new inputs, with eager passes and synchronizations
    between the replays."""
    s = state(1)
    everything(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = everything(s)
    for seed in (1, 20, 30, 40):
        new = state(seed)
        for k in s:
            s[k].copy_(new[k])
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert same(got, everything(new)), seed
        assert same(got, everything(s)), seed
        torch.cuda.synchronize()


def test_workspaces_of_the_caller():
    h, w, targets, gloss = case(200, 400, 64, torch.bfloat16)
    t = targets.to(DEV)
    n = ops.zs_xent_workspace_bytes(h.data_ptr(), 64, w.data_ptr(), 64, 200, 400, 64, 1)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)  # NaN wherever it is read unwritten
    want = ops.linear_xent(h, w, t)
    got = ops.linear_xent(h, w, t, workspace=ws)
    assert same(got, want)
    ws.fill_(255)
    assert same(ops.linear_xent_backward(h, w, t, want[1], gloss.to(DEV), workspace=ws),
                ops.linear_xent_backward(h, w, t, want[1], gloss.to(DEV)))
    d = rows(200, 64, torch.bfloat16, 3)
    ws = torch.full((ops.zs_embed_backward_bytes(200, 400, 64),), 255, dtype=torch.uint8, device=DEV)
    assert same([ops.embed_backward(d, t, 400, workspace=ws)], [ops.embed_backward(d, t, 400)])
    ws = torch.full((ops.zs_norm_backward_bytes(200, 64),), 255, dtype=torch.uint8, device=DEV)
    one, rstd = torch.ones(64, dtype=torch.bfloat16, device=DEV), torch.ones(200, device=DEV)
    assert same(ops.norm_backward(d, h, one, rstd, workspace=ws), ops.norm_backward(d, h, one, rstd))


def test_xent_refuses():
    h, w, targets, gloss = case(20, 40, 64, torch.bfloat16)
    t, f = targets.to(DEV), gloss.to(DEV)
    for call in (lambda: ops.linear_xent(h.float(), w.float(), t), lambda: ops.linear_xent(h, w.half(), t),
                 lambda: ops.linear_xent(h, w[:, :32], t), lambda: ops.linear_xent(h, w, t[:3]),
                 lambda: ops.linear_xent(h, w, t.float()), lambda: ops.linear_xent(h, w, t.cpu()),
                 lambda: ops.linear_xent(h.t(), w, t), lambda: ops.linear_xent(h, w.cpu(), t),
                 lambda: ops.linear_xent(h, w, t, workspace=f.view(torch.uint8)),
                 lambda: ops.linear_xent(h, w[:0], t),
                 lambda: ops.linear_xent_backward(h, w, t, f.double(), f),
                 lambda: ops.linear_xent_backward(h, w, t, f, f[:3]),
                 lambda: ops.linear_xent_backward(h, w, t, f, f, out=w),
                 lambda: ops.linear_xent_backward(h, w, t, f, f, weight_grad_out=w.float())):
        with pytest.raises(ValueError):
            call()
