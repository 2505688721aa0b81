"""Model operators that make the gradient contributions a ZeRO shard step reads.

Four operators on torch tensors, run by the HIP kernels of libzeroshard.so: the
token embedding, the root-mean-square norm with the residual's addition and an
8-bit output, activations held in 8 bits (alone and under a gated unit), and the
softmax cross entropy of a linear head.  Every C entry point of
include/zeroshard_ops.h is exposed under the same name; the functions on tensors
below check what the kernels will stream over, allocate outputs and workspace
with torch, and enqueue on torch's current stream of the tensors' device.

There is no autograd here: forward and backward are separate calls, and what the
backward reads is what the forward returned.  Tensors that require a gradient are
read like any other, and results carry no history.  Matrices are 2-D with adjacent
elements in a row and any row stride of at least the width; ``out=`` arguments
take such views too, so a gradient can be written straight into a contribution
buffer of ZeroShard.  They must not overlap what the call reads or the call's other
outputs, except where its description allows an input itself.  Arguments the kernels
could not read or write so are refused with ValueError before anything is enqueued.

The 8-bit form: codes as torch.float8_e4m3fn or torch.float8_e5m2, and one
power-of-two scale (torch.float8_e8m0fnu) for each group of 32, 64 or 128
neighbouring elements; the value is code * scale.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _check, _f32, _i32, _i64, _sig, _sz, _vp

ZS_F32, ZS_BF16, ZS_F16 = 0, 1, 2
ZS_E4M3, ZS_E5M2 = 0, 1
ZS_SILU, ZS_GELU = 0, 1

_INT = ctypes.c_int
_embed_forward = _sig("zs_embed_forward", _INT, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _i64,
                      _f32, _i32, _i32, _vp)
_embed_backward_bytes = _sig("zs_embed_backward_bytes", _sz, _i64, _i64, _i64)
_embed_backward = _sig("zs_embed_backward", _INT, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _i64,
                       _i64, _f32, _i32, _i32, _i32, _i32, _vp, _sz, _vp)
_norm_forward = _sig("zs_norm_forward", _INT, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64,
                     _vp, _vp, _vp, _i64, _i64, _f32, _i32, _i32, _i32, _vp)
_norm_backward_bytes = _sig("zs_norm_backward_bytes", _sz, _i64, _i64)
_norm_backward = _sig("zs_norm_backward", _INT, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp,
                      _i64, _vp, _i64, _i64, _i32, _i32, _vp, _sz, _vp)
_act8_pack = _sig("zs_act8_pack", _INT, _vp, _i64, _vp, _vp, _i64, _i64, _i32, _i32, _i32, _vp)
_act8_unpack = _sig("zs_act8_unpack", _INT, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _i32, _i32,
                    _vp)
_glu_forward = _sig("zs_glu_forward", _INT, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _i32,
                    _i32, _i32, _i32, _vp)
_glu_backward = _sig("zs_glu_backward", _INT, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _i64,
                     _i64, _i32, _i32, _i32, _i32, _vp)
_xent_workspace_bytes = _sig("zs_xent_workspace_bytes", _sz, _vp, _i64, _vp, _i64, _i64, _i64,
                             _i64, _i32)
_xent_forward = _sig("zs_xent_forward", _INT, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64,
                     _i64, _i32, _i32, _vp, _sz, _vp)
_xent_backward = _sig("zs_xent_backward", _INT, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64,
                      _vp, _i64, _i64, _i64, _i64, _i32, _i32, _vp, _sz, _vp)

EXPORTED = ["zs_embed_forward", "zs_embed_backward_bytes", "zs_embed_backward", "zs_norm_forward",
            "zs_norm_backward_bytes", "zs_norm_backward", "zs_act8_pack", "zs_act8_unpack",
            "zs_glu_forward", "zs_glu_backward", "zs_xent_workspace_bytes", "zs_xent_forward",
            "zs_xent_backward"]


# The C entry points under their names: arguments as in zeroshard_ops.h, device
# addresses as ints (0 or None: NULL); negative codes raise ZeroShardError.


def zs_embed_forward(*args) -> None:
    _check(_embed_forward(*args))


def zs_embed_backward_bytes(n_tokens: int, vocab: int, width: int) -> int:
    return int(_embed_backward_bytes(n_tokens, vocab, width))


def zs_embed_backward(*args) -> None:
    _check(_embed_backward(*args))


def zs_norm_forward(*args) -> None:
    _check(_norm_forward(*args))


def zs_norm_backward_bytes(rows: int, width: int) -> int:
    return int(_norm_backward_bytes(rows, width))


def zs_norm_backward(*args) -> None:
    _check(_norm_backward(*args))


def zs_act8_pack(*args) -> None:
    _check(_act8_pack(*args))


def zs_act8_unpack(*args) -> None:
    _check(_act8_unpack(*args))


def zs_glu_forward(*args) -> None:
    _check(_glu_forward(*args))


def zs_glu_backward(*args) -> None:
    _check(_glu_backward(*args))


def zs_xent_workspace_bytes(*args) -> int:
    return int(_xent_workspace_bytes(*args))


def zs_xent_forward(*args) -> None:
    _check(_xent_forward(*args))


def zs_xent_backward(*args) -> None:
    _check(_xent_backward(*args))


# ---------------------------------------------------------------- checks

_DTYPES = {torch.float32: ZS_F32, torch.bfloat16: ZS_BF16, torch.float16: ZS_F16}
_HALVES = {torch.bfloat16: ZS_BF16, torch.float16: ZS_F16}
_CODES = {"e4m3": (ZS_E4M3, torch.float8_e4m3fn), "e5m2": (ZS_E5M2, torch.float8_e5m2)}
_CODE_OF = {torch.float8_e4m3fn: ZS_E4M3, torch.float8_e5m2: ZS_E5M2}
_SCALE = torch.float8_e8m0fnu
_ACTS = {"silu": ZS_SILU, "gelu": ZS_GELU}
_ID_BYTES = {torch.int64: 8, torch.int32: 4}


def _matrix(t, name, dtype=None, device=None, rows=None, width=None):
    """A 2-D tensor the kernels can read: its row stride."""
    if t.dim() != 2:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected 2")
    if device is None:
        if not t.is_cuda:
            raise ValueError(f"{name}: on {t.device}, expected a GPU")
    elif t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    r, w = t.shape
    if (rows is not None and r != rows) or (width is not None and w != width):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected "
                         f"({'any' if rows is None else rows}, {'any' if width is None else width})")
    s, e = t.stride()
    if r <= 1 or w == 0:
        s = max(s, w)
    if (e != 1 and w > 1) or s < w:
        raise ValueError(f"{name}: strides {t.stride()}: elements of a row must be adjacent and "
                         "rows must not overlap")
    return s


def _vector(t, name, dtypes, device, n):
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected ({n},)")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name}: not contiguous")


def _dtype(t, name, allowed=_DTYPES):
    d = allowed.get(t.dtype)
    if d is None:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {tuple(allowed)}")
    return d


def _pick(table, key, name):
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{name}: {key!r}, expected one of {tuple(table)}") from None


def _group(group):
    if group not in (32, 64, 128):
        raise ValueError(f"group: {group!r}, expected 32, 64 or 128")
    return group


# The current stream's handle: the raw query, where torch has it, costs a
# twentieth of making a Stream object, which a call on a few rows would notice.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(device, entry, *args):
    """Calls a C entry point on torch's current stream of the device, with that
    device current."""
    index = device.index
    if torch.cuda.current_device() == index:
        rc = entry(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = entry(*args, _raw_stream(index))
    if rc < 0:
        _check(rc)


def _extent(t):
    """(address, rows, bytes from row to row, bytes of a row) of a matrix, or of a
    contiguous tensor as one row."""
    e = t.element_size()
    if t.dim() == 2 and t.shape[0] > 1:
        return t.data_ptr(), t.shape[0], t.stride(0) * e, t.shape[1] * e
    return t.data_ptr(), 1, t.numel() * e, t.numel() * e


def _overlap(a, b):
    """Whether two tensors share a byte: rows of views side by side in one buffer do not."""
    pa, na, sa, wa = _extent(a)
    pb, nb, sb, wb = _extent(b)
    if not wa or not wb or pa + (na - 1) * sa + wa <= pb or pb + (nb - 1) * sb + wb <= pa:
        return False
    if na > nb:
        pa, na, sa, wa, pb, nb, sb, wb = pb, nb, sb, wb, pa, na, sa, wa
    if na == 1:
        at = torch.tensor([pa - pb], device="cpu")
    else:
        at = torch.arange(na, dtype=torch.int64, device="cpu") * sa + (pa - pb)
    # of each row of a: the first of b's rows that ends behind its beginning
    row = torch.div(at - wb, sb, rounding_mode="floor").add_(1).clamp_(min=0)
    return bool(((row < nb) & (row * sb < at + wa)).any())


def _apart(out, name, allowed, others):
    """Refuses an output that overlaps an input; it may be one of `allowed` itself."""
    for t in allowed:
        if t is not None and _extent(t) != _extent(out):
            others = (*others, t)
    for t in others:
        if t is not None and _overlap(out, t):
            raise ValueError(f"{name}: overlaps another buffer of the call")


def _workspace(given, nbytes, device):
    if nbytes == 0:
        raise ValueError("a size is out of the range the operator takes")
    if given is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if given.dtype != torch.uint8 or given.device != device or not given.is_contiguous():
        raise ValueError(f"workspace: expected contiguous uint8 on {device}")
    if given.numel() < nbytes or given.data_ptr() % 256:
        raise ValueError(f"workspace: {given.numel()} bytes at {given.data_ptr():#x}, the call "
                         f"needs {nbytes} at a multiple of 256")
    return given


def _ids(ids, device):
    if ids.dtype not in _ID_BYTES:
        raise ValueError(f"ids: dtype {ids.dtype}, expected one of {tuple(_ID_BYTES)}")
    if ids.device != device:
        raise ValueError(f"ids: on {ids.device}, expected {device}")
    if not ids.is_contiguous():
        raise ValueError("ids: not contiguous")
    return _ID_BYTES[ids.dtype]


# ---------------------------------------------------------------- embedding


def embed(table, ids, scale=1.0, vocab_start=0, out=None):
    """scale * table[ids - vocab_start], one row a token; ids outside the table give
    zeros.  ids: int32 or int64 of any shape; the result has that shape and the
    table's width last (out=: a matrix with one row a token)."""
    stride = _matrix(table, "table")
    dev = table.device
    dt = _dtype(table, "table")
    nb = _ids(ids, dev)
    vocab, width = table.shape
    n = ids.numel()
    if out is None:
        out = torch.empty(*ids.shape, width, dtype=table.dtype, device=dev)
        out_stride = width
    else:
        out_stride = _matrix(out, "out", table.dtype, dev, n, width)
        _apart(out, "out", (), (table, ids))
    _run(dev, _embed_forward, table.data_ptr(), stride, ids.data_ptr(), out.data_ptr(), out_stride,
         n, vocab, width, vocab_start, scale, dt, nb)
    return out


def embed_backward(grad_out, ids, vocab, scale=1.0, vocab_start=0, out=None, out_dtype=None,
                   accumulate=False, workspace=None):
    """The table's gradient [vocab, width]: scale * the sum of grad_out's rows by id,
    in a fixed order.  grad_out: ids' shape and the width last.  out= takes the
    gradient (a contribution buffer's view); with accumulate=True it is added to
    what out holds, and rows without tokens are left alone."""
    if grad_out.dim() != 2:
        if not grad_out.is_contiguous() or grad_out.shape[:-1] != ids.shape:
            raise ValueError("grad_out: expected ids' shape and the width, contiguous")
        grad_out = grad_out.view(-1, grad_out.shape[-1])
    n = ids.numel()
    stride = _matrix(grad_out, "grad_out", rows=n)
    dev = grad_out.device
    dt = _dtype(grad_out, "grad_out")
    nb = _ids(ids, dev)
    width = grad_out.shape[1]
    if out is None:
        if accumulate:
            raise ValueError("accumulate: needs out, the gradient to add to")
        out = torch.empty(vocab, width, dtype=out_dtype or grad_out.dtype, device=dev)
        out_stride = width
    else:
        out_stride = _matrix(out, "out", out_dtype, dev, vocab, width)
        _apart(out, "out", (), (grad_out, ids))
    if out.dtype not in (grad_out.dtype, torch.float32):
        raise ValueError(f"out: dtype {out.dtype}, expected {grad_out.dtype} or torch.float32")
    ws = _workspace(workspace, _embed_backward_bytes(n, vocab, width), dev)
    _run(dev, _embed_backward, grad_out.data_ptr(), stride, ids.data_ptr(), out.data_ptr(),
         out_stride, n, vocab, width, vocab_start, scale, dt, _DTYPES[out.dtype], nb,
         int(accumulate), ws.data_ptr(), ws.numel())
    return out


# ---------------------------------------------------------------- norm


class NormOut(NamedTuple):
    """What norm returns; the fields that were not asked for are None (sum without a
    residual is x itself)."""
    y: Optional[torch.Tensor]
    sum: torch.Tensor
    rstd: torch.Tensor
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


def norm(x, weight, residual=None, eps=1e-6, code=None, group=128, want_y=True):
    """y = s / sqrt(mean(s^2) + eps) * weight with s = x + residual, row by row.
    y in x's dtype where want_y; in 8 bits (codes, scales) where code is "e4m3" or
    "e5m2".  rstd [rows] and s are what norm_backward reads."""
    xs = _matrix(x, "x")
    dev = x.device
    dt = _dtype(x, "x")
    rows, width = x.shape
    _vector(weight, "weight", (x.dtype,), dev, width)
    s, rs, ss = x, 0, 0
    if residual is not None:
        rs = _matrix(residual, "residual", x.dtype, dev, rows, width)
        s = torch.empty(rows, width, dtype=x.dtype, device=dev)
        ss = width
    y = torch.empty(rows, width, dtype=x.dtype, device=dev) if want_y else None
    rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    codes = scales = None
    cd = 0
    if code is not None:
        cd, ct = _pick(_CODES, code, "code")
        _group(group)
        codes = torch.empty(rows, width, dtype=ct, device=dev)
        scales = torch.empty(rows, -(-width // group), dtype=_SCALE, device=dev)
    if rows:
        _run(dev, _norm_forward, x.data_ptr(), xs, residual.data_ptr() if residual is not None else
             None, rs, weight.data_ptr(), s.data_ptr() if residual is not None else None, ss,
             y.data_ptr() if want_y else None, width, codes.data_ptr() if code is not None else
             None, scales.data_ptr() if code is not None else None, rstd.data_ptr(), rows, width,
             eps, dt, cd, group)
    return NormOut(y, s, rstd, codes, scales)


def norm_backward(grad_y, sum, weight, rstd, grad_sum=None, out=None, weight_grad_out=None,
                  weight_grad_dtype=None, workspace=None):
    """(grad_x, grad_weight) of norm: grad_x is the gradient of x and of the residual
    alike, with grad_sum (the gradient that reaches s by the residual path) added.
    grad_weight in the weight's dtype, or fp32 with weight_grad_dtype=torch.float32.
    out may be grad_y, sum or grad_sum itself."""
    gs = _matrix(grad_y, "grad_y")
    dev = grad_y.device
    dt = _dtype(grad_y, "grad_y")
    rows, width = grad_y.shape
    ss = _matrix(sum, "sum", grad_y.dtype, dev, rows, width)
    _vector(weight, "weight", (grad_y.dtype,), dev, width)
    _vector(rstd, "rstd", (torch.float32,), dev, rows)
    ds = 0
    if grad_sum is not None:
        ds = _matrix(grad_sum, "grad_sum", grad_y.dtype, dev, rows, width)
    if out is None:
        out = torch.empty(rows, width, dtype=grad_y.dtype, device=dev)
        os_ = width
    else:
        os_ = _matrix(out, "out", grad_y.dtype, dev, rows, width)
        _apart(out, "out", (grad_y, sum, grad_sum), (weight, rstd))
    if weight_grad_out is None:
        weight_grad_out = torch.empty(width, dtype=weight_grad_dtype or grad_y.dtype, device=dev)
    else:
        _vector(weight_grad_out, "weight_grad_out",
                (weight_grad_dtype,) if weight_grad_dtype else (grad_y.dtype, torch.float32), dev,
                width)
        _apart(weight_grad_out, "weight_grad_out", (), (grad_y, sum, weight, rstd, grad_sum, out))
    if weight_grad_out.dtype not in (grad_y.dtype, torch.float32):
        raise ValueError(f"weight_grad_dtype: {weight_grad_out.dtype}, expected {grad_y.dtype} or "
                         "torch.float32")
    ws = _workspace(workspace, _norm_backward_bytes(rows, width), dev)
    _run(dev, _norm_backward, grad_y.data_ptr(), gs, sum.data_ptr(), ss, weight.data_ptr(),
         rstd.data_ptr(), grad_sum.data_ptr() if ds else None, ds, out.data_ptr(), os_,
         weight_grad_out.data_ptr(), rows, width, dt, _DTYPES[weight_grad_out.dtype], ws.data_ptr(),
         ws.numel())
    return out, weight_grad_out


# ---------------------------------------------------------------- 8-bit activations


def pack8(x, code="e4m3", group=128):
    """(codes, scales) of a matrix in the 8-bit form."""
    xs = _matrix(x, "x")
    dev = x.device
    dt = _dtype(x, "x")
    cd, ct = _pick(_CODES, code, "code")
    _group(group)
    rows, width = x.shape
    codes = torch.empty(rows, width, dtype=ct, device=dev)
    scales = torch.empty(rows, -(-width // group), dtype=_SCALE, device=dev)
    if rows:
        _run(dev, _act8_pack, x.data_ptr(), xs, codes.data_ptr(), scales.data_ptr(), rows, width,
             dt, cd, group)
    return codes, scales


def _checkpoint(codes, scales, rows, width, halves, group):
    """The format of a checkpoint of `halves` matrices side by side; its codes and
    scales must lie as pack8 and glu wrote them."""
    cd = _dtype(codes, "codes", _CODE_OF)
    dev = codes.device
    if not codes.is_cuda:
        raise ValueError(f"codes: on {dev}, expected a GPU")
    if tuple(codes.shape) != (rows, halves * width) or not codes.is_contiguous():
        raise ValueError(f"codes: shape {tuple(codes.shape)}, expected ({rows}, {halves * width}), "
                         "contiguous")
    groups = -(-width // group)
    want = (rows, groups) if halves == 1 else (rows, halves, groups)
    if scales.dtype != _SCALE or scales.device != dev:
        raise ValueError(f"scales: {scales.dtype} on {scales.device}, expected {_SCALE} on {dev}")
    if tuple(scales.shape) != want or not scales.is_contiguous():
        raise ValueError(f"scales: shape {tuple(scales.shape)}, expected {want}, contiguous")
    return cd


def unpack8(codes, scales, dtype, group=128, out=None):
    """The values of an 8-bit checkpoint (pack8's or norm's), rounded once to dtype."""
    dt = _pick(_DTYPES, dtype, "dtype")
    _group(group)
    if codes.dim() != 2:
        raise ValueError(f"codes: {codes.dim()} dimensions, expected 2")
    rows, width = codes.shape
    cd = _checkpoint(codes, scales, rows, width, 1, group)
    dev = codes.device
    if out is None:
        out = torch.empty(rows, width, dtype=dtype, device=dev)
        stride = width
    else:
        stride = _matrix(out, "out", dtype, dev, rows, width)
        _apart(out, "out", (), (codes, scales))
    if rows:
        _run(dev, _act8_unpack, codes.data_ptr(), scales.data_ptr(), out.data_ptr(), stride, rows,
             width, dt, cd, group)
    return out


def glu(gate_up, act="silu", code="e4m3", group=128):
    """(out, codes, scales): out = act(gate) * up of gate_up = [gate | up], and
    gate_up itself in the 8-bit form for glu_backward (scales [rows, 2, groups]).
    code=None keeps nothing (codes and scales are None)."""
    gs = _matrix(gate_up, "gate_up")
    dev = gate_up.device
    dt = _dtype(gate_up, "gate_up")
    a = _pick(_ACTS, act, "act")
    rows, both = gate_up.shape
    if both % 2 or both == 0:
        raise ValueError(f"gate_up: width {both}, expected two halves")
    width = both // 2
    _group(group)
    out = torch.empty(rows, width, dtype=gate_up.dtype, device=dev)
    codes = scales = None
    cd = 0
    if code is not None:
        cd, ct = _pick(_CODES, code, "code")
        codes = torch.empty(rows, both, dtype=ct, device=dev)
        scales = torch.empty(rows, 2, -(-width // group), dtype=_SCALE, device=dev)
    if rows:
        _run(dev, _glu_forward, gate_up.data_ptr(), gs, out.data_ptr(), width, codes.data_ptr() if
             code is not None else None, scales.data_ptr() if code is not None else None, rows,
             width, dt, a, cd, group)
    return out, codes, scales


def glu_backward(grad_out, codes, scales, act="silu", group=128, want_out=False, out=None):
    """(grad_gate_up, out): the gated unit's gradient from its 8-bit checkpoint, and
    with want_out its output again, from the same checkpoint (None otherwise).
    out= takes grad_gate_up."""
    gs = _matrix(grad_out, "grad_out")
    dev = grad_out.device
    dt = _dtype(grad_out, "grad_out")
    a = _pick(_ACTS, act, "act")
    _group(group)
    rows, width = grad_out.shape
    cd = _checkpoint(codes, scales, rows, width, 2, group)
    if codes.device != dev:
        raise ValueError(f"codes: on {codes.device}, expected {dev}")
    if out is None:
        out = torch.empty(rows, 2 * width, dtype=grad_out.dtype, device=dev)
        os_ = 2 * width
    else:
        os_ = _matrix(out, "out", grad_out.dtype, dev, rows, 2 * width)
        _apart(out, "out", (), (grad_out, codes, scales))
    again = torch.empty(rows, width, dtype=grad_out.dtype, device=dev) if want_out else None
    if rows:
        _run(dev, _glu_backward, grad_out.data_ptr(), gs, codes.data_ptr(), scales.data_ptr(),
             out.data_ptr(), os_, again.data_ptr() if want_out else None, width, rows, width, dt, a,
             cd, group)
    return out, again


# ---------------------------------------------------------------- cross entropy


def _xent_args(hidden, weight, targets):
    hs = _matrix(hidden, "hidden")
    dev = hidden.device
    dt = _dtype(hidden, "hidden", _HALVES)
    ws = _matrix(weight, "weight", hidden.dtype, dev, width=hidden.shape[1])
    _vector(targets, "targets", _ID_BYTES, dev, hidden.shape[0])
    return hs, ws, dev, dt, _ID_BYTES[targets.dtype]


def linear_xent(hidden, weight, targets, workspace=None):
    """(loss, lse), both fp32 [tokens]: the softmax cross entropy of hidden @
    weight.T against targets, without the logits.  A target outside the vocabulary
    (-100, say) marks a token that does not count; its loss is 0."""
    hs, wstride, dev, dt, nb = _xent_args(hidden, weight, targets)
    tokens, width = hidden.shape
    vocab = weight.shape[0]
    loss = torch.empty(tokens, dtype=torch.float32, device=dev)
    lse = torch.empty(tokens, dtype=torch.float32, device=dev)
    h, w = hidden.data_ptr(), weight.data_ptr()
    ws = _workspace(workspace, _xent_workspace_bytes(h, hs, w, wstride, tokens, vocab, width, 0),
                    dev)
    _run(dev, _xent_forward, h, hs, w, wstride, targets.data_ptr(), loss.data_ptr(), lse.data_ptr(),
         tokens, vocab, width, dt, nb, ws.data_ptr(), ws.numel())
    return loss, lse


def linear_xent_backward(hidden, weight, targets, lse, grad_loss, out=None, weight_grad_out=None,
                         want_hidden=True, want_weight=True, workspace=None):
    """(grad_hidden, grad_weight) of linear_xent for grad_loss [tokens] (fp32; 1/n for
    a mean over n tokens, times the loss scale where gradients are fp16).  What is
    not wanted is None.  out may be hidden itself."""
    hs, wstride, dev, dt, nb = _xent_args(hidden, weight, targets)
    tokens, width = hidden.shape
    vocab = weight.shape[0]
    _vector(lse, "lse", (torch.float32,), dev, tokens)
    _vector(grad_loss, "grad_loss", (torch.float32,), dev, tokens)
    gh = gw = None
    ghs = gws = width
    if want_hidden:
        gh = out
        if gh is None:
            gh = torch.empty(tokens, width, dtype=hidden.dtype, device=dev)
        else:
            ghs = _matrix(gh, "out", hidden.dtype, dev, tokens, width)
            _apart(gh, "out", (hidden,), (weight, targets, lse, grad_loss))
    if want_weight:
        gw = weight_grad_out
        if gw is None:
            gw = torch.empty(vocab, width, dtype=hidden.dtype, device=dev)
        else:
            gws = _matrix(gw, "weight_grad_out", hidden.dtype, dev, vocab, width)
            _apart(gw, "weight_grad_out", (), (hidden, weight, targets, lse, grad_loss, gh))
    h, w = hidden.data_ptr(), weight.data_ptr()
    ws = _workspace(workspace, _xent_workspace_bytes(h, hs, w, wstride, tokens, vocab, width, 1),
                    dev)
    _run(dev, _xent_backward, h, hs, w, wstride, targets.data_ptr(), lse.data_ptr(),
         grad_loss.data_ptr(), gh.data_ptr() if want_hidden else None, ghs, gw.data_ptr() if
         want_weight else None, gws, tokens, vocab, width, dt, nb, ws.data_ptr(), ws.numel())
    return gh, gw
