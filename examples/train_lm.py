"""A small language model trained on one GPU with the operators and the shard step.

    python examples/train_lm.py [--steps 200]

Token ids go through the embedding, layers of norm and gated unit on a residual
stream, a last norm and the cross entropy of a head that shares the embedding's
table.  What the backward pass needs is kept in 8 bits: the norms' outputs (codes
and scales, for the weight gradient of the product that follows) and the gated
units' inputs.  The products between the operators are torch's.

Every weight is a view of the shard's 16-bit parameters and every gradient is
written into a view of a contribution buffer, one buffer a micro-batch; the step
then averages the contributions, clips by the global norm and updates the fp32
state and the weights.  The data are a noisy successor function on the
vocabulary, so that the loss has something to fall towards.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sharded_optimizer_step_zero_amd import ZeroShard, ops, zs_plan_tensor_slice  # noqa: E402


class Model:
    """Shapes, the shard that owns the weights, and views into its buffers."""

    def __init__(self, vocab=1000, width=256, inner=704, layers=2, micro_batches=2, device="cuda",
                 seed=0):
        self.vocab, self.width, self.inner, self.layers = vocab, width, inner, layers
        self.shapes = [(vocab, width)]
        for _ in range(layers):
            self.shapes += [(width,), (2 * inner, width), (width, inner)]
        self.shapes += [(width,)]
        numel = [torch.Size(s).numel() for s in self.shapes]
        decay = [len(s) == 2 for s in self.shapes]
        self.shard = ZeroShard(numel, decay, M=micro_batches, device=device, grad_buffers=True)
        self.weights = self.views(self.shard.param)
        self.grads = [self.views(g) for g in self.shard.grads]
        self.scale = width ** 0.5
        g = torch.Generator(device=self.shard.device).manual_seed(seed)
        for view, s in zip(self.views(self.shard.master), self.shapes):
            if len(s) == 1:
                view.fill_(1.0)
            else:
                view.copy_(torch.randn(s, generator=g, device=view.device) * s[1] ** -0.5)
        self.shard.param.copy_(self.shard.master)

    def views(self, flat):
        out = []
        for i, s in enumerate(self.shapes):
            at, _, n = zs_plan_tensor_slice(self.shard.plan, i)
            assert n == torch.Size(s).numel()  # one rank owns every tensor whole
            out.append(flat[at:at + n].view(s))
        return out

    def micro_batch(self, j, ids, targets, weight):
        """One forward and backward pass: the gradients of sum(loss * weight) into
        contribution j, and the tokens' losses."""
        w, gr = self.weights, self.grads[j]
        table = w[0]
        # forward
        stream = ops.embed(table, ids, scale=self.scale)
        branch, kept = None, []
        for k in range(self.layers):
            wn, wgu, wd = w[1 + 3 * k:4 + 3 * k]
            n = ops.norm(stream, wn, residual=branch, code="e4m3")
            out, codes, scales = ops.glu(n.y @ wgu.t())
            kept.append((n.sum, n.rstd, n.codes, n.scales, codes, scales))
            stream, branch = n.sum, out @ wd.t()
        last = ops.norm(stream, w[-1], residual=branch)
        loss, lse = ops.linear_xent(last.y, table, targets)
        # backward
        dy, _ = ops.linear_xent_backward(last.y, table, targets, lse, weight, weight_grad_out=gr[0])
        d, _ = ops.norm_backward(dy, last.sum, w[-1], last.rstd, weight_grad_out=gr[-1])
        for k in reversed(range(self.layers)):
            wn, wgu, wd = w[1 + 3 * k:4 + 3 * k]
            dwn, dwgu, dwd = gr[1 + 3 * k:4 + 3 * k]
            total, rstd, y8, y8s, codes, scales = kept[k]
            dgu, out = ops.glu_backward(d @ wd, codes, scales, want_out=True)
            torch.mm(d.t(), out, out=dwd)
            torch.mm(dgu.t(), ops.unpack8(y8, y8s, dgu.dtype), out=dwgu)
            d, _ = ops.norm_backward(dgu @ wgu, total, wn, rstd, grad_sum=d, weight_grad_out=dwn)
        ops.embed_backward(d, ids, self.vocab, scale=self.scale, out=gr[0], accumulate=True)
        return loss


def batch(model, tokens, generator):
    """Ids with a language's frequencies, and their successors: a fixed function of
    the id for nine tokens in ten; some tokens are padding."""
    dev = model.shard.device
    u = torch.rand(tokens, generator=generator, device=dev)
    ids = ((model.vocab + 1.0) ** u).long().clamp_(1, model.vocab) - 1
    targets = (ids * 7 + 3) % model.vocab
    noise = torch.rand(tokens, generator=generator, device=dev)
    other = torch.randint(0, model.vocab, (tokens,), generator=generator, device=dev)
    targets = torch.where(noise < 0.1, other, targets)
    targets[:: 50] = -100
    return ids, targets


def train(steps=200, tokens=2048, micro_batches=2, lr=2e-3, seed=0, report=None, **shape):
    """The mean loss of every step."""
    model = Model(micro_batches=micro_batches, seed=seed, **shape)
    g = torch.Generator(device=model.shard.device).manual_seed(seed + 1)
    losses = []
    for step in range(1, steps + 1):
        total, count = 0.0, 0
        for j in range(micro_batches):
            ids, targets = batch(model, tokens, g)
            counts = targets >= 0
            # the step averages the contributions, so each carries its own mean
            weight = counts.float() / counts.sum()
            total = total + model.micro_batch(j, ids, targets, weight).sum()
            count = count + counts.sum()
        model.shard.step(model.shard.grads, lr=lr, beta1=0.9, beta2=0.95, eps=1e-8,
                         weight_decay=0.01, step=step, max_grad_norm=1.0)
        losses.append(total / count)
        if report and (step == 1 or step % report == 0):
            print(f"step {step}: loss {float(losses[-1]):.4f}", flush=True)
    out = [float(x) for x in losses]
    model.shard.close()
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--tokens", type=int, default=2048, help="of one micro-batch")
    a = ap.parse_args()
    train(a.steps, a.tokens, report=20)
