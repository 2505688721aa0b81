"""The order in which the embedding's gradient adds: tokens of an id in order of t within
fixed runs of sorted tokens, then the runs' parts in theirs.  Sums whose last bits depend
on the order, equal bit for bit."""
import numpy as np
import pytest
import torch

from sharded_optimizer_step_zero_amd import ops

from test_gpu_ops_embed import DEV, gen, make_ids, rows

pytestmark = pytest.mark.gpu


def in_order(dout, ids, vocab, run):
    """The sums in fp32, one addition at a time; tokens are sorted by their id's last eight
    bits, then by the rest."""
    d = dout.cpu().float().numpy()
    v = ids.numpy()
    order = [t for t in np.argsort((v & 255) * vocab + (v >> 8), kind="stable") if 0 <= v[t] < vocab]
    out = np.zeros((vocab, d.shape[1]), np.float32)
    parts = {}
    for place, t in enumerate(order):
        parts.setdefault(v[t], {}).setdefault(place // run, []).append(t)
    for i, by_run in parts.items():
        sums = []
        for r in sorted(by_run):
            s = np.zeros(d.shape[1], np.float32)
            for t in by_run[r]:
                s = s + d[t]
            sums.append(s)
        total = sums[0]
        for s in sums[1:]:
            total = total + s
        out[i] = total
    return torch.from_numpy(out)


@pytest.mark.parametrize("tokens, vocab, kind, run", [
    (5000, 40, "random", 8), (5000, 3000, "skewed", 8), (4000, 5, "same", 8), (3000, 2000, "bucket", 8),
    (70_000, 300, "skewed", 32), (20_000, 70_000, "skewed", 32), (12_288, 900, "random", 8),
    (12_289, 900, "random", 32)])
def test_sums_are_added_in_order(tokens, vocab, kind, run):
    ids = make_ids(kind, tokens, vocab, 4)
    dout = rows(tokens, 8, torch.float32, 5)
    want = in_order(dout, ids, vocab, run)
    for dtype in (torch.int64, torch.int32):
        got = ops.embed_backward(dout, ids.to(dtype).to(DEV), vocab)
        assert torch.equal(got.cpu(), want)
    assert int((want != torch.zeros(vocab, 8).index_add_(0, ids.clamp(0, vocab - 1)[(ids >= 0) & (ids < vocab)].flip(0),
                                                         dout.cpu()[(ids >= 0) & (ids < vocab)].flip(0))).sum()) > 0
