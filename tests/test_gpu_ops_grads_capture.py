"""Making a list of gradients copies from the host, which a capture does not hold: it is refused
there, and the capture goes on."""
import pytest
import torch

from sharded_optimizer_step_zero_amd import ops

pytestmark = pytest.mark.gpu


def test_a_list_made_during_a_capture_is_refused():
    t = [torch.full((n,), 2.0, device="cuda") for n in (50, 4096, 10000)]
    rows = ops.GradList(t)
    want = ops.grad_sumsq(rows)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in (lambda: ops.GradList(t), lambda: ops.clip_grads(t, 1.0), lambda: ops.grad_sumsq(t)):
            with pytest.raises(ValueError, match="before a capture"):
                call()
        got = ops.grad_sumsq(rows)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and all(bool((x == 2.0).all()) for x in t)
