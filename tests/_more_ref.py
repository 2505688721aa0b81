"""The layer norm, the 4-bit form with its product, the preference loss and the clipping of many
gradients in float64 on the CPU, from their formulas.  Bounds count roundings (see _ops_ref)."""
import math

import torch

from _ops_ref import E, f64

FOUR = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


# ------------------------------------------------------------------ layer norm


def layer_norm(s, weight, bias, eps):
    """(y, mean, rstd, the magnitude that y's roundings are relative to)"""
    mean = s.mean(1)
    d = s - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + eps)
    p = d * rstd[:, None] * weight
    b = bias if bias is not None else torch.zeros_like(weight)
    return p + b, mean, rstd, p.abs() + b.abs()


def layer_norm_grad(dy, s, weight, mean, rstd, ds=None):
    """(dx, dw, db, and the magnitudes of dx, dw, db)"""
    h = (s - mean[:, None]) * rstd[:, None]
    g = dy * weight
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    size = rstd[:, None] * (g.abs() + g.abs().mean(1, keepdim=True)
                            + h.abs() * (g * h).abs().mean(1, keepdim=True))
    if ds is not None:
        dx, size = dx + ds, size + ds.abs()
    return dx, (dy * h).sum(0), dy.sum(0), size, (dy * h).abs().sum(0), dy.abs().sum(0)


# ------------------------------------------------------------------ 4-bit form


def pack4(x):
    """(values of the codes, the scales' exponents + 127) [rows, groups, 32] and [rows, groups]; a
    group that is not finite has byte 255 and codes 0.  x in float64."""
    rows, d = x.shape
    n = -(-d // 32)
    p = torch.zeros(rows, n * 32, dtype=torch.float64)
    p[:, :d] = x
    p = p.view(rows, n, 32)
    fine = torch.isfinite(p).all(2)
    q = torch.where(fine[:, :, None], p, torch.zeros(()).double())
    amax = q.abs().amax(2)
    e = torch.full_like(amax, -127)
    for k in range(-126, 128):  # the least e that holds the group
        e = torch.where(amax > 6 * 2.0 ** (k - 1), torch.full_like(e, k), e)
    q = q * torch.exp2(-e)[:, :, None]
    # the nearest value, of two the one with the even code
    gap = (q.abs()[..., None] - FOUR).abs()
    least = gap.amin(-1, keepdim=True)
    at = torch.where(gap == least, torch.tensor([0, 9, 1, 9, 2, 9, 3, 9]) + torch.where(
        torch.arange(8) % 2 == 0, 0, 1), torch.full((8,), 99)).argmin(-1)
    byte = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return FOUR[at] * torch.where(q < 0, -1.0, 1.0), byte


def values4(codes, byte, width):
    s = torch.exp2(byte.double() - 127)
    s[byte == 255] = math.nan
    return (codes * s[:, :, None]).view(codes.shape[0], -1)[:, :width]


def read4(c):
    """(values of the codes, scale bytes) as pack4 above gives them, of a Codes4; the scales of
    groups that do not exist have to be 1."""
    b = c.codes.cpu().view(torch.uint8).long()
    rows, groups = b.shape[0], b.shape[1] // 16
    nib = torch.stack([b & 15, b >> 4], -1).view(rows, groups, 32)
    v = FOUR[nib & 7] * torch.where(nib >= 8, -1.0, 1.0)
    s = c.scales.cpu().view(torch.uint8)
    plain = s.permute(1, 0, 3, 2).reshape(rows, -1)
    assert plain.shape[1] == -(-groups // 16) * 16
    assert bool((plain[:, groups:] == 127).all())
    return v, plain[:, :groups]


# ------------------------------------------------------------------ preference loss


def prefer(loss, ref, offsets, mask, beta, kind, margin=0.0, smoothing=0.0, average=False, grad=None):
    """(loss, rewards, margins, lengths, sum of magnitudes of each sequence, slope and, with grad,
    the tokens' gradient)"""
    o = [min(max(int(v), 0), loss.numel()) for v in offsets]
    n = len(o) - 1
    counts = torch.ones(loss.numel(), dtype=torch.bool) if mask is None else mask.cpu().bool()
    d = f64(loss) - (0 if ref is None else f64(ref))
    big = f64(loss).abs() + (0 if ref is None else f64(ref).abs())
    a, size, lengths = torch.zeros(n).double(), torch.zeros(n).double(), torch.zeros(n, dtype=torch.int64)
    for i in range(n):
        at = torch.arange(o[i], max(o[i], o[i + 1]))
        at = at[counts[at]]
        lengths[i] = at.numel()
        over = max(1, at.numel()) if average else 1
        a[i], size[i] = -d[at].sum() / over, big[at].sum() / over
    r = (a * beta).view(-1, 2)
    m = r[:, 0] - r[:, 1] - margin
    sp = torch.nn.functional.softplus
    if kind == "sigmoid":
        out = (1 - smoothing) * sp(-m) + smoothing * sp(m)
        slope = -(1 - smoothing) * torch.sigmoid(-m) + smoothing * torch.sigmoid(m)
    elif kind == "hinge":
        out, slope = (1 - m).clamp(min=0), torch.where(m < 1, -1.0, 0.0).double()
    else:
        out, slope = (m - 0.5) ** 2 / beta ** 2, 2 * (m - 0.5) / beta ** 2
    g = None
    if grad is not None:
        g = torch.zeros(loss.numel()).double()
        for i in range(n):
            at = torch.arange(o[i], max(o[i], o[i + 1]))
            at = at[counts[at]]
            over = max(1, at.numel()) if average else 1
            g[at] = float(slope[i // 2] * f64(grad)[i // 2]) * beta / over * (1 if i % 2 else -1)
    return out, r, m, lengths.view(-1, 2), (size * beta).view(-1, 2), slope, g


# ------------------------------------------------------------------ many gradients


def clip(tensors, max_norm):
    """(norm, clipped values)"""
    norm = math.sqrt(math.fsum(float((f64(t) ** 2).sum()) for t in tensors))
    c = min(1.0, max_norm / (norm + 1e-6)) if not math.isnan(norm) else math.nan
    return norm, [f64(t) * c for t in tensors]


__all__ = ["E", "layer_norm", "layer_norm_grad", "pack4", "values4", "read4", "prefer", "clip"]
