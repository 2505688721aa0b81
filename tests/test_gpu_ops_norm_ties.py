"""The norm's 8-bit output where one bit decides: codes next to a tie and groups next to a
border of the scale are those of the products in fp64."""
import pytest
import torch

import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops

from test_gpu_ops_embed import DEV, TYPES, gen

pytestmark = pytest.mark.gpu


def near_ties(code, group, width, seed):
    """One fp32 row and a weight for which every element's scaled value lies within a few
    units of a tie of its code (normal and subnormal codes), one element of each group
    giving the scale."""
    g = gen(seed)
    s = torch.randn(1, width, generator=g)
    s = torch.where(s.abs() < 0.1, torch.full_like(s, 0.7), s)
    r = R.norm(s.double(), torch.ones(width, dtype=torch.float64), 1e-6)[1]
    bits, low = (3, -6) if code == "e4m3" else (2, -14)
    # ties: an odd multiple of half a step, of a binade or below the least normal
    e = torch.randint(low - 1, R.TOP[code] - 1, (width,), generator=g)
    m = torch.randint(0, 2 ** bits, (width,), generator=g).double()
    tie = torch.where(e < low, (m + 0.5) * 2.0 ** (low - bits), (2 ** bits + m + 0.5) * torch.exp2(e.double() - bits))
    tie[::group] = 1.5 * 2.0 ** R.TOP[code]  # gives the scale 1
    w = (tie / (s[0].double() * r[0])).float()
    units = torch.randint(-3, 4, (width,), generator=g)
    units[::group] = 0
    return s, (w.view(torch.int32) + units.int()).view(torch.float32)


def exact_codes(y, code):
    """y (fp64, scale 1) rounded to the code's grid, ties to even."""
    bits, low = (3, -6) if code == "e4m3" else (2, -14)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** (low - 1)))).clamp(min=low)
    step = torch.exp2(e - bits)
    return torch.round(y / step) * step


@pytest.mark.parametrize("code", ["e4m3", "e5m2"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("width", [500, 4096, 65536])
def test_codes_next_to_a_tie(code, group, width):
    """Equal to those of the products in fp64, every one."""
    for seed in range(8):
        s, w = near_ties(code, group, width, seed)
        out = ops.norm(s.to(DEV), w.to(DEV), code=code, group=group, want_y=False)
        assert (R.byte_of(out.scales) == 127).all()
        y = R.norm(s.double(), w.double(), 1e-6)[0]
        got, want = R.f64(out.codes.float()), exact_codes(y, code)
        assert torch.equal(got, want), (seed, int((got != want).sum()))


@pytest.mark.parametrize("code", ["e4m3", "e5m2"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_groups_next_to_a_border(code, group):
    """A group's largest value within a few units of 1.75 times a power of two."""
    width = 65536
    for seed in range(4):
        g = gen(seed)
        s = torch.randn(1, width, generator=g)
        s = torch.where(s.abs() < 0.1, torch.full_like(s, 0.7), s)
        r = R.norm(s.double(), torch.ones(width, dtype=torch.float64), 1e-6)[1]
        w = torch.randn(width, generator=g) * 0.1
        at = torch.arange(0, width, group) + torch.randint(0, group, (width // group,), generator=g)
        e = torch.randint(2, 17, (at.numel(),), generator=g).double()
        w[at] = (1.75 * torch.exp2(e) / (s[0, at].double() * r[0])).float()
        units = torch.randint(-3, 4, (at.numel(),), generator=g).int()
        w[at] = (w[at].view(torch.int32) + units).view(torch.float32)
        out = ops.norm(s.to(DEV), w.to(DEV), code=code, group=group, want_y=False)
        y = R.norm(s.double(), w.double(), 1e-6)[0]
        amax = y.abs().view(-1, group).amax(1)
        byte = R.byte_of(out.scales)[0].double()
        top = 1.75 * torch.exp2(byte - 127 + R.TOP[code])
        assert ((amax <= top) & (amax > top / 2)).all(), seed


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("code", ["e4m3", "e5m2"])
def test_codes_of_many_values(dtype, code):
    """Groups of which most elements have subnormal codes: bytes and codes all equal."""
    n, width, group = 3000, 2000, 64
    size = torch.full((width,), 0.3 if code == "e4m3" else 1e-5)
    size[::group] = 1e4  # gives the scale
    for residual in (False, True):
        x = (torch.randn(n, width, generator=gen(1)) * size).to(dtype)
        r = (torch.randn(n, width, generator=gen(2)) * size).to(dtype) if residual else None
        w = (1 + 0.1 * torch.randn(width, generator=gen(3))).to(dtype)
        out = ops.norm(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV), code=code, group=group,
                       want_y=False)
        s = out.sum.double()
        y = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * w.to(DEV).double()
        scale = torch.exp2(out.scales.view(torch.uint8).double() - 127)
        pad = torch.zeros(n, scale.shape[1] * group, dtype=torch.float64, device=DEV)
        pad[:, :width] = y.abs()
        amax, top = pad.view(n, -1, group).amax(2), 1.75 * 2.0 ** R.TOP[code] * scale
        assert ((amax <= top) & (amax > top / 2)).all()
        want = exact_codes(y / scale.repeat_interleave(group, 1)[:, :width], code)
        got = out.codes.float().double()
        assert torch.equal(got, want), int((got != want).sum())
