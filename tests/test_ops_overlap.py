"""Whether two views share memory, against sets of their bytes."""
import random

import pytest
import torch

from sharded_optimizer_step_zero_amd import ops


def cells(t):
    base = torch.arange(t.element_size())
    at = torch.zeros(t.shape, dtype=torch.int64)
    for d, (n, s) in enumerate(zip(t.shape, t.stride())):
        shape = [1] * t.dim()
        shape[d] = n
        at = at + (torch.arange(n) * s).view(shape)
    return set((at.reshape(-1, 1) * t.element_size() + t.data_ptr() + base).reshape(-1).tolist())


def test_views_of_one_buffer():
    rng = random.Random(1)
    buffer = torch.zeros(4000, dtype=torch.uint8)
    dtypes = [torch.uint8, torch.bfloat16, torch.float32]

    def view():
        flat = buffer.view(rng.choice(dtypes))
        if rng.random() < 0.2:
            n = rng.randrange(0, 300)
            at = rng.randrange(0, flat.numel() - n + 1)
            return flat[at:at + n]
        stride = rng.choice([7, 16, 24, 40, 61])
        width = rng.randrange(0, stride + 1)
        rows = rng.randrange(0, max(2, min(25, flat.numel() // stride)))
        at = rng.randrange(0, flat.numel() - rows * stride + 1)
        return flat[at:at + rows * stride].view(rows, stride)[:, :width]
    seen = set()
    for _ in range(6000):
        a, b = view(), view()
        want = bool(cells(a) & cells(b))
        assert ops._overlap(a, b) == want, (a.shape, a.stride(), a.data_ptr(), b.shape, b.stride(), b.data_ptr())
        close = a.dim() == b.dim() == 2 and a.numel() > 0 and b.numel() > 0
        seen.add((want, close and a.stride(0) * a.element_size() == b.stride(0) * b.element_size()))
    assert len(seen) == 4


def test_halves_of_a_row_are_apart():
    both = torch.zeros(5, 64)
    assert not ops._overlap(both[:, :32], both[:, 32:])
    assert ops._overlap(both[:, :33], both[:, 32:])
    assert not ops._overlap(both[:2], both[2:]) and ops._overlap(both, both[4])


def test_one_row_is_itself_whatever_its_stride():
    """A row's stride to a next one that is not there does not make it another buffer."""
    a = torch.zeros(4, 64)
    ops._apart(a[:1], "out", (a.view(2, 128)[:1, :64],), ())
    ops._apart(a[:, :32], "out", (a[:, :32],), ())
    for other in (a[:1, :63], a[:1, 1:], a[:2]):
        with pytest.raises(ValueError, match="overlaps"):
            ops._apart(a[:1], "out", (other,), ())


def test_the_default_device_takes_no_part():
    a = torch.zeros(40, 64)
    was = torch.get_default_device()
    try:
        torch.set_default_device("meta")
        assert not ops._overlap(a[:, :32], a[:, 32:]) and ops._overlap(a[:, :33], a[:, 32:])
        assert ops._overlap(a, a[3]) and not ops._overlap(a[:, :8], a[3, 8:])
    finally:
        torch.set_default_device(was)
