"""A list of gradients that is dropped while work on it is still queued on another stream than the
one it was made on: its table's memory is not given away before that work is done."""
import pytest
import torch

from sharded_optimizer_step_zero_amd import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("made_on_a_side_stream", [False, True])
@pytest.mark.parametrize("call", ["clip", "sumsq", "clip by a given sum"])
@pytest.mark.parametrize("again", [False, True])
def test_a_list_dropped_behind_queued_work(made_on_a_side_stream, call, again):
    t = [torch.full((n,), 2.0, device="cuda") for n in (50, 4096, 10000, 7)]
    count = sum(x.numel() for x in t)
    given = torch.full((), 4.0 * count, dtype=torch.float64, device="cuda")
    home, other = torch.cuda.current_stream(), torch.cuda.Stream()
    if made_on_a_side_stream:
        home, other = other, home
    torch.cuda.synchronize()
    with torch.cuda.stream(home):
        rows = ops.GradList(t)
        at, nbytes = rows.table.data_ptr(), rows.table.numel()
    home.synchronize()
    with torch.cuda.stream(other):
        if again:  # a call before, whose work is done
            ops.grad_sumsq(rows)
            other.synchronize()
        torch.cuda._sleep(200_000_000)  # a tenth of a second or so
        if call == "sumsq":
            got = ops.grad_sumsq(rows)
        else:
            got = ops.clip_grads(rows, 1.0, sumsq=given if call != "clip" else None)
        under_way = not other.query()
    del rows
    with torch.cuda.stream(home):
        # nothing is written to these
        new = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(64)]
    assert under_way and not other.query()
    assert all(x.data_ptr() != at for x in new)
    torch.cuda.synchronize()
    if call == "sumsq":
        assert float(got) == 4.0 * count
    else:
        norm = 2.0 * count ** 0.5
        assert abs(float(got) - norm) <= norm * 2.0 ** -50
        # the factor and the product are rounded to fp32; 1e-6 of a norm of 238 is less than another rounding
        assert all(bool(((x.double() - 2.0 / norm).abs() <= 3 * 2.0 ** -24 * 2.0 / norm).all()) for x in t)


def test_on_its_own_stream_the_table_is_given_back_at_once():
    t = [torch.ones(3000, device="cuda")]
    torch.cuda.synchronize()
    rows = ops.GradList(t)
    at, nbytes = rows.table.data_ptr(), rows.table.numel()
    ops.clip_grads(rows, 1e6)
    del rows
    assert torch.empty(nbytes, dtype=torch.uint8, device="cuda").data_ptr() == at
    torch.cuda.synchronize()


def test_a_graph_of_a_list_that_was_made_on_another_stream():
    t = [torch.full((n,), 2.0, device="cuda") for n in (50, 4096, 10000)]
    out = [torch.empty_like(x) for x in t]
    rows = ops.GradList(t, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want_norm = ops.clip_grads(rows, 1.0)
    side.synchronize()
    want = [x.clone() for x in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        norm = ops.clip_grads(rows, 1.0)
    for scale in (1.0, 3.0, 0.5):
        for x, o in zip(t, out):
            x.fill_(2.0 * scale)
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        # the same direction, the same length: two roundings to fp32 on either side, and 1e-6 of a norm
        # of 119 or more
        assert abs(float(norm) - float(want_norm) * scale) <= float(norm) * 2.0 ** -40
        assert all(bool(((o - w).abs() <= w.abs() * 5 * 2.0 ** -24).all()) for o, w in zip(out, want))
