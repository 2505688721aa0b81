"""The operators together: a training step on pairs of sequences, with layer norms, products in 4
bits, the preference loss of the head's losses and gradients that are clipped into a
contribution of the shard step.  Its gradients are those of the same model in float64."""
import math

import pytest
import torch

import _more_ref as M
from sharded_optimizer_step_zero_amd import ZeroShard, ops, zs_plan_tensor_slice

pytestmark = pytest.mark.gpu
VOCAB, WIDTH, INNER = 500, 256, 320
SHAPES = [(VOCAB, WIDTH), (WIDTH,), (WIDTH,), (2 * INNER, WIDTH), (WIDTH, INNER), (WIDTH,), (WIDTH,)]


class Model:
    def __init__(self):
        self.shard = ZeroShard([math.prod(s) for s in SHAPES], [len(s) == 2 for s in SHAPES], M=1, grad_buffers=True)
        g = torch.Generator(device="cuda").manual_seed(1)
        for v, s in zip(self.views(self.shard.master), SHAPES):
            v.copy_(torch.randn(s, generator=g, device="cuda") * (s[-1] ** -0.5 if len(s) == 2 else 0.1))
        for i in (1, 5):
            self.views(self.shard.master)[i].add_(1.0)
        self.shard.param.copy_(self.shard.master)
        self.weights = self.views(self.shard.param)
        bf, f32 = torch.bfloat16, torch.float32
        self.grads = [torch.empty(s, dtype=bf if len(s) == 2 else f32, device="cuda") for s in SHAPES]
        self.list = ops.GradList(self.grads, out=self.views(self.shard.grads[0]))

    def views(self, flat):
        at = [zs_plan_tensor_slice(self.shard.plan, i) for i in range(len(SHAPES))]
        return [flat[a:a + n].view(s) for (a, _, n), s in zip(at, SHAPES)]

    def gradients(self, ids, targets, ref, offsets, mask):
        table, w1, b1, up, down, w2, b2 = self.weights
        d_table, d_w1, d_b1, d_up, d_down, d_w2, d_b2 = self.grads
        n_tok = ids.numel()
        x = ops.embed(table, ids, scale=16.0)
        n = ops.layer_norm(x, w1, b1, code="e2m1")
        out, codes, scales = ops.glu(ops.linear4(ops.Codes4(n.codes, n.scales, WIDTH), ops.pack4(up)))
        out_rows, out_columns = ops.pack4(out, want="both")
        last = ops.layer_norm(ops.linear4(out_rows, ops.pack4(down)), w2, b2, residual=x)
        loss, lse = ops.linear_xent(last.y, table, targets)
        pref = ops.preference_loss(loss, ref, offsets, beta=0.2, mask=mask)
        pairs = pref.loss.numel()
        each = ops.preference_loss_backward(pref, offsets, torch.full((pairs,), 1.0 / pairs, device="cuda"), n_tok,
                                            beta=0.2, mask=mask)
        dy, _ = ops.linear_xent_backward(last.y, table, targets, lse, each, weight_grad_out=d_table)
        d, _, _ = ops.layer_norm_backward(dy, last.sum, w2, last.mean, last.rstd, weight_grad_out=d_w2, bias_grad_out=d_b2)
        rows, columns = ops.pack4(d, want="both")
        ops.linear4(columns, out_columns, out=d_down)
        d_gu, _ = ops.glu_backward(ops.linear4(rows, ops.pack4(down, want="columns")), codes, scales)
        rows, columns = ops.pack4(d_gu, want="both")
        ops.linear4(columns, ops.pack4(n.y, want="columns"), out=d_up)
        dn = ops.linear4(rows, ops.pack4(up, want="columns"))
        d, _, _ = ops.layer_norm_backward(dn, x, w1, n.mean, n.rstd, grad_sum=d, weight_grad_out=d_w1, bias_grad_out=d_b1)
        ops.embed_backward(d, ids, VOCAB, scale=16.0, out=d_table, accumulate=True)
        return pref, loss


def batch():
    g = torch.Generator(device="cuda").manual_seed(2)
    t, pairs = 700, 6
    ids = torch.randint(0, VOCAB, (t,), generator=g, device="cuda")
    targets = torch.randint(0, VOCAB, (t,), generator=g, device="cuda")
    mask = torch.rand(t, generator=g, device="cuda") < 0.8
    targets[~mask] = -100
    ref = torch.where(mask, 6.2 + torch.randn(t, generator=g, device="cuda") * 0.2, torch.zeros(t, device="cuda"))
    cut = torch.randint(0, t - 20, (2 * pairs - 1,), generator=g, device="cuda").sort().values
    offsets = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), t - 20)])
    return ids, targets, ref, offsets, mask


class Through(torch.autograd.Function):
    """y = q(x) q(w)^T of the values in 4 bits; its gradients from dy, w and x packed along the axis
    that is summed over."""

    @staticmethod
    def forward(ctx, x, w):
        ctx.save_for_backward(x, w)
        return four(x) @ four(w).t()

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        t = lambda v: v.t().contiguous()  # noqa: E731
        return four(dy) @ four(t(w)).t(), four(t(dy)) @ four(t(x)).t()


def four(x):
    c, b = M.pack4(x.detach())
    return M.values4(c, b, x.shape[1])


def test_gradients_against_float64():
    m = Model()
    ids, targets, ref, offsets, mask = batch()
    pref, loss = m.gradients(ids, targets, ref, offsets, mask)
    w = [v.detach().cpu().double().requires_grad_() for v in m.weights]
    ids, targets, ref, mask, o = ids.cpu(), targets.cpu(), ref.cpu().double(), mask.cpu(), offsets.tolist()

    def norm(x, a, b):
        d = x - x.mean(1, keepdim=True)
        return d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * a + b

    x = w[0][ids] * 16.0
    gu = Through.apply(norm(x, w[1], w[2]), w[3])
    gate, up = gu[:, :INNER], gu[:, INNER:]
    h = norm(x + Through.apply(gate * torch.sigmoid(gate) * up, w[4]), w[5], w[6])
    lp = torch.nn.functional.cross_entropy(h @ w[0].t(), targets, ignore_index=-100, reduction="none")
    a = torch.stack([-(lp - ref)[o[i]:o[i + 1]][mask[o[i]:o[i + 1]]].sum() for i in range(len(o) - 1)]).view(-1, 2) * 0.2
    want = torch.nn.functional.softplus(a[:, 1] - a[:, 0])
    want.mean().backward()
    # A value that is off by 2^-9 of itself gets another code where it lies that near a tie, of
    # which there is one for each quarter of its size or so: two in a hundred codes move by a
    # third, 2^-4 of a packed operand's size, and an 8-bit checkpoint is off by 2^-5.  No gradient has more
    # than five packed operands and one checkpoint on its way.
    bound = 5 * 2.0 ** -4 + 2.0 ** -5
    for got, v in zip(m.grads, w):
        got = got.cpu().double()
        assert float((got - v.grad).norm() / v.grad.norm()) < bound
    # a token's loss of about 6 from activations that are off by 2^-4 of their branch
    assert float((loss.cpu().double() - lp.detach()).abs().max()) < 1.0
    m.shard.close()


def test_a_step_and_its_clip():
    """The contribution is the clipped gradients, the step moves every weight that has one, and all
    of it comes out the same twice."""
    runs = []
    for _ in range(2):
        m = Model()
        m.gradients(*batch())
        norm = ops.clip_grads(m.list, 0.05)
        want_norm, want = M.clip(m.grads, 0.05)
        assert math.isclose(float(norm), want_norm, rel_tol=1e-13) and want_norm > 0.05
        for got, v in zip(m.views(m.shard.grads[0]), want):
            got = got.cpu().double()
            assert bool(((got - v).abs() <= v.abs() * 2.0 ** -8 * 1.01 + 1e-38).all())
        before = m.shard.param.clone()
        m.shard.step(m.shard.grads, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, step=1)
        moved = [bool((a != b).any()) for a, b in zip(m.views(before), m.weights)]
        assert all(moved)
        runs.append([m.shard.grads[0].clone(), m.shard.param.clone(), m.shard.master.clone()])
        m.shard.close()
    assert all(torch.equal(a, b) for a, b in zip(*runs))
