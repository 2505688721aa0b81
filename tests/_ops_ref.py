"""The model operators in float64 on the CPU, from their formulas, and the error
bounds their kernels are held to.

u(t) is half a unit in the last place of a value in [1, 2) of type t: one rounding
to t is off by at most u(t) relative (or half the least subnormal).  Bounds count
roundings; E = 2^-24 is fp32's.
"""
import math

import torch

E = 2.0 ** -24
TOP = {"e4m3": 8, "e5m2": 15}
CODE_DTYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
CODE_U = {"e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
CODE_SUB = {"e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}  # half the least subnormal


def u(dtype):
    return torch.finfo(dtype).eps / 2


def sub(dtype):
    """Half the least subnormal."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().cpu().double()


def close(got, want, bound, what):
    """|got - want| <= bound element by element; non-finite values agree."""
    got = f64(got)
    assert got.shape == want.shape, what
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    d = (got - want).abs()[fine]
    b = (bound if torch.is_tensor(bound) else torch.full_like(want, bound)).expand_as(want)[fine]
    bad = d > b
    if bad.any():
        k = int((d - b).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {d.numel()} off, worst {float(d[k]):.3g} "
                             f"against {float(b[k]):.3g}")


def rounded(want, dtype, roundings=0.0):
    """Bound of a value with so many fp32 roundings and one to dtype."""
    return want.abs() * (u(dtype) + roundings * E) * (1 + 2.0 ** -7) + sub(dtype) + sub(torch.float32)


# ------------------------------------------------------------------ embedding


def embed(table, ids, scale, start=0):
    v = ids.cpu().long().reshape(-1) - start
    ok = (v >= 0) & (v < table.shape[0])
    out = torch.zeros(v.numel(), table.shape[1], dtype=torch.float64)
    out[ok] = f64(table)[v[ok]] * scale
    return out


def embed_grad(dout, ids, vocab, scale, start=0):
    """(the gradient, sum of magnitudes, tokens of each id)"""
    v = ids.cpu().long().reshape(-1) - start
    ok = (v >= 0) & (v < vocab)
    d = f64(dout).reshape(v.numel(), -1)[ok]
    total = torch.zeros(vocab, d.shape[1], dtype=torch.float64)
    size = torch.zeros_like(total)
    total.index_add_(0, v[ok], d)
    size.index_add_(0, v[ok], d.abs())
    return total * scale, size * abs(scale), torch.bincount(v[ok], minlength=vocab).double()[:, None]


# ------------------------------------------------------------------ norm


def norm(s, weight, eps):
    rstd = 1 / torch.sqrt((s * s).mean(1) + eps)
    return s * rstd[:, None] * weight, rstd


def norm_grad(dy, s, weight, rstd, ds=None):
    h = s * rstd[:, None]
    wdy = dy * weight
    dot = (wdy * h).mean(1, keepdim=True)
    dx = rstd[:, None] * (wdy - h * dot)
    size = rstd[:, None] * (wdy.abs() + h.abs() * (wdy * h).abs().mean(1, keepdim=True))
    if ds is not None:
        dx, size = dx + ds, size + ds.abs()
    return dx, (dy * h).sum(0), size, (dy * h).abs().sum(0)


# ------------------------------------------------------------------ 8-bit form


def pack(x, code, group):
    """(codes, scale bytes) bit for bit; x fp32 or narrower."""
    x = x.detach().cpu().float()
    rows, d = x.shape
    n = -(-d // group)
    p = torch.zeros(rows, n * group)
    p[:, :d] = x
    p = p.view(rows, n, group)
    amax = p.double().abs().amax(2)
    fine = torch.isfinite(p).all(2)
    a = torch.where(fine, amax, torch.zeros_like(amax))
    e = torch.full_like(a, -127)
    for k in range(-126, 128):  # the least e that holds the group
        e = torch.where(a > 1.75 * 2.0 ** (TOP[code] + k - 1), torch.full_like(e, k), e)
    q = torch.where(fine[:, :, None], p.double() * torch.exp2(-e)[:, :, None], torch.zeros(()).double())
    codes = q.float().to(CODE_DTYPE[code]).view(rows, n * group)[:, :d].contiguous()
    byte = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return codes, byte


def unpack(codes, byte, group):
    s = torch.exp2(byte.cpu().double() - 127)
    s[byte.cpu() == 255] = math.nan
    d = codes.shape[-1]
    return codes.cpu().float().double() * s.repeat_interleave(group, -1)[..., :d]


def byte_of(scales):
    return scales.view(torch.uint8).cpu()


# ------------------------------------------------------------------ gated unit


def act(x, kind):
    """(act, slope, relative error in units of E of the sigmoid, slope's magnitude)"""
    if kind == "silu":
        s = 1 / (1 + torch.exp(-x))
        arg, t = x, s * (1 - s)
        return x * s, s + x * t, 2 * arg.abs() + 8, s + (x * t).abs()
    k = math.sqrt(2 / math.pi)
    z2 = 2 * k * (x + 0.044715 * x ** 3)
    s = 1 / (1 + torch.exp(-z2))
    t = s * (1 - s)
    r = 2 * k * x * t * (1 + 0.134145 * x * x)
    return x * s, s + r, 8 * z2.abs() + 12, s + r.abs()


# ------------------------------------------------------------------ cross entropy


def xent(h, w, targets, gloss=None):
    """loss, lse, the logits' error bound and, with gloss, dh, dw and G."""
    h, w = f64(h), f64(w)
    targets = targets.cpu().long()
    live = (targets >= 0) & (targets < w.shape[0])
    logits = h @ w.t().contiguous()
    size = h.abs() @ w.abs().t().contiguous()
    lse = torch.logsumexp(logits, 1)
    at = targets.clamp(0, w.shape[0] - 1)[:, None]
    loss = torch.where(live, lse - logits.gather(1, at)[:, 0], torch.zeros_like(lse))
    err = (h.shape[1] + 2) * 2 * E * size  # fp32 sums, an addition off by a unit
    if gloss is None:
        return loss, lse, logits, err
    g = torch.exp(logits - lse[:, None])
    g.scatter_add_(1, at, -torch.ones_like(lse)[:, None])
    g = torch.where(live[:, None], g * f64(gloss)[:, None], torch.zeros(()).double())
    hh = torch.where(live[:, None], h, torch.zeros(()).double())
    return loss, lse, logits, err, g, g @ w, g.t().contiguous() @ hh, live, hh, w
