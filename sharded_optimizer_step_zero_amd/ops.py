"""Model operators that make the gradient contributions a ZeRO shard step reads.

Operators on torch tensors, run by the HIP kernels of libzeroshard.so: the
token embedding, the root-mean-square norm with the residual's addition and an
8-bit output, the layer norm with an output in 16, 8 or 4 bits, activations held
in 8 bits (alone and under a gated unit), matrices in 4 bits and their product, the
softmax cross entropy of a linear head, the preference loss on its tokens' losses, and
the clipping of many tensors by their global norm.  Every C entry point of
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
neighbouring elements; the value is code * scale.  The 4-bit form (Codes4) has
groups of 32.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _check, _f32, _i32, _i64, _sig, _sz, _vp

ZS_F32, ZS_BF16, ZS_F16 = 0, 1, 2
ZS_E4M3, ZS_E5M2, ZS_E2M1 = 0, 1, 2
ZS_SILU, ZS_GELU = 0, 1
ZS_SIGMOID, ZS_HINGE, ZS_SQUARED = 0, 1, 2



class GradTensor(ctypes.Structure):
    """zs_grad_tensor: seven 64-bit words, the types in the last one's halves."""
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("width", ctypes.c_int64), ("grad_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


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
_layer_norm_forward = _sig("zs_layer_norm_forward", _INT, _vp, _i64, _vp, _i64, _vp, _vp, _vp,
                           _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _f32, _i32, _i32,
                           _i32, _vp)
_layer_norm_backward_bytes = _sig("zs_layer_norm_backward_bytes", _sz, _i64, _i64)
_layer_norm_backward = _sig("zs_layer_norm_backward", _INT, _vp, _i64, _vp, _i64, _vp, _vp, _vp,
                            _vp, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _i32, _i32, _vp, _sz, _vp)
_mx4_pack = _sig("zs_mx4_pack", _INT, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp)
_mx4_unpack = _sig("zs_mx4_unpack", _INT, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp)
_mx4_product = _sig("zs_mx4_product", _INT, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32,
                    _vp)
_mx4_linear_bytes = _sig("zs_mx4_linear_bytes", _sz, _i64, _i64)
_mx4_linear = _sig("zs_mx4_linear", _INT, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32,
                   _i32, _vp, _sz, _vp)
_prefer_workspace_bytes = _sig("zs_prefer_workspace_bytes", _sz, _i64, _i64)
_prefer_forward = _sig("zs_prefer_forward", _INT, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                       _i64, _f32, _f32, _f32, _i32, _i32, _i32, _vp, _sz, _vp)
_prefer_backward = _sig("zs_prefer_backward", _INT, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                        _f32, _f32, _i32, _i32, _i32, _vp)
_grads_pieces = _sig("zs_grads_pieces", _i64, _vp, _i64)
_grads_table = _sig("zs_grads_table", _INT, _vp, _i64, _vp, _sz)
_grads_workspace_bytes = _sig("zs_grads_workspace_bytes", _sz, _i64)
_grads_sumsq = _sig("zs_grads_sumsq", _INT, _vp, _i64, _vp, _vp, _sz, _vp)
_grads_clip = _sig("zs_grads_clip", _INT, _vp, _i64, _f32, _vp, _vp, _vp, _sz, _vp)

EXPORTED = ["zs_embed_forward", "zs_embed_backward_bytes", "zs_embed_backward", "zs_norm_forward",
            "zs_norm_backward_bytes", "zs_norm_backward", "zs_act8_pack", "zs_act8_unpack",
            "zs_glu_forward", "zs_glu_backward", "zs_xent_workspace_bytes", "zs_xent_forward",
            "zs_xent_backward", "zs_layer_norm_forward", "zs_layer_norm_backward_bytes",
            "zs_layer_norm_backward", "zs_mx4_pack", "zs_mx4_unpack", "zs_mx4_product",
            "zs_mx4_linear_bytes", "zs_mx4_linear",
            "zs_prefer_workspace_bytes", "zs_prefer_forward", "zs_prefer_backward",
            "zs_grads_pieces", "zs_grads_table", "zs_grads_workspace_bytes", "zs_grads_sumsq",
            "zs_grads_clip"]


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


def zs_layer_norm_forward(*args) -> None:
    _check(_layer_norm_forward(*args))


def zs_layer_norm_backward_bytes(rows: int, width: int) -> int:
    return int(_layer_norm_backward_bytes(rows, width))


def zs_layer_norm_backward(*args) -> None:
    _check(_layer_norm_backward(*args))


def zs_mx4_pack(*args) -> None:
    _check(_mx4_pack(*args))


def zs_mx4_unpack(*args) -> None:
    _check(_mx4_unpack(*args))


def zs_mx4_product(*args) -> None:
    _check(_mx4_product(*args))


def zs_mx4_linear_bytes(tokens: int, width: int) -> int:
    return int(_mx4_linear_bytes(tokens, width))


def zs_mx4_linear(*args) -> None:
    _check(_mx4_linear(*args))


def zs_prefer_workspace_bytes(tokens: int, pairs: int) -> int:
    return int(_prefer_workspace_bytes(tokens, pairs))


def zs_prefer_forward(*args) -> None:
    _check(_prefer_forward(*args))


def zs_prefer_backward(*args) -> None:
    _check(_prefer_backward(*args))


def _grad_array(tensors):
    return (GradTensor * max(1, len(tensors)))(*tensors)


def zs_grads_pieces(tensors) -> int:
    """tensors: GradTensor records."""
    return int(_check(_grads_pieces(_grad_array(tensors), len(tensors))))


def zs_grads_table(tensors, table: int, table_bytes: int) -> None:
    _check(_grads_table(_grad_array(tensors), len(tensors), table, table_bytes))


def zs_grads_workspace_bytes(pieces: int) -> int:
    return int(_grads_workspace_bytes(pieces))


def zs_grads_sumsq(*args) -> None:
    _check(_grads_sumsq(*args))


def zs_grads_clip(*args) -> None:
    _check(_grads_clip(*args))


# ---------------------------------------------------------------- checks

_DTYPES = {torch.float32: ZS_F32, torch.bfloat16: ZS_BF16, torch.float16: ZS_F16}
_HALVES = {torch.bfloat16: ZS_BF16, torch.float16: ZS_F16}
_CODES = {"e4m3": (ZS_E4M3, torch.float8_e4m3fn), "e5m2": (ZS_E5M2, torch.float8_e5m2)}
_CODE_OF = {torch.float8_e4m3fn: ZS_E4M3, torch.float8_e5m2: ZS_E5M2}
_SCALE = torch.float8_e8m0fnu
_FOUR = torch.float4_e2m1fn_x2
_NORM_CODES = {**_CODES, "e2m1": (ZS_E2M1, _FOUR)}
_KINDS = {"sigmoid": ZS_SIGMOID, "hinge": ZS_HINGE, "squared": ZS_SQUARED}
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
    if t.dim() == 1 and t.shape[0] == n and t.dtype in dtypes and t.device == device and (
            n <= 1 or t.stride(0) == 1):
        return
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
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(device, entry, *args):
    """Calls a C entry point on torch's current stream of the device, with that
    device current."""
    index = device.index
    if _current_device() == index:
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


# ---------------------------------------------------------------- layer norm


class LayerNormOut(NamedTuple):
    """What layer_norm returns; the fields that were not asked for are None (sum without a
    residual is x itself)."""
    y: Optional[torch.Tensor]
    sum: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


def layer_norm(x, weight, bias=None, residual=None, eps=1e-5, code=None, group=None, want_y=True):
    """y = (s - mean(s)) / sqrt(mean((s - mean(s))^2) + eps) * weight + bias with s = x +
    residual, row by row.  y in x's dtype where want_y; (codes, scales) in 8 bits where code is
    "e4m3" or "e5m2" (groups of 128 unless group says 32 or 64), in the 4-bit form where it is
    "e2m1": Codes4(codes, scales, width) is an operand of linear4.  mean and rstd [rows] and s
    are what layer_norm_backward reads."""
    xs = _matrix(x, "x")
    dev = x.device
    dt = _dtype(x, "x")
    rows, width = x.shape
    _vector(weight, "weight", (x.dtype,), dev, width)
    if bias is not None:
        _vector(bias, "bias", (x.dtype,), dev, width)
    s, rs, ss = x, 0, 0
    if residual is not None:
        rs = _matrix(residual, "residual", x.dtype, dev, rows, width)
        s = torch.empty(rows, width, dtype=x.dtype, device=dev)
        ss = width
    y = torch.empty(rows, width, dtype=x.dtype, device=dev) if want_y else None
    stats = torch.empty(2, rows, dtype=torch.float32, device=dev)
    mean, rstd = stats.unbind()
    codes = scales = None
    cd = 0
    if code is not None:
        cd, ct = _pick(_NORM_CODES, code, "code")
    if cd == ZS_E2M1:
        if group not in (None, 32):
            raise ValueError(f"group: {group!r}, the 4-bit form has groups of 32")
        group = 32
        codes, scales = _empty4(rows, width, dev)
    elif code is not None:
        group = _group(128 if group is None else group)
        codes = torch.empty(rows, width, dtype=ct, device=dev)
        scales = torch.empty(rows, -(-width // group), dtype=_SCALE, device=dev)
    if rows:
        _run(dev, _layer_norm_forward, x.data_ptr(), xs, residual.data_ptr() if residual is not None
             else None, rs, weight.data_ptr(), bias.data_ptr() if bias is not None else None,
             s.data_ptr() if residual is not None else None, ss, y.data_ptr() if want_y else None,
             width, codes.data_ptr() if code is not None else None, scales.data_ptr() if code is not
             None else None, mean.data_ptr(), rstd.data_ptr(), rows, width, eps, dt, cd, group or 32)
    return LayerNormOut(y, s, mean, rstd, codes, scales)


def layer_norm_backward(grad_y, sum, weight, mean, rstd, grad_sum=None, out=None,
                        weight_grad_out=None, bias_grad_out=None, weight_grad_dtype=None,
                        want_bias=True, workspace=None):
    """(grad_x, grad_weight, grad_bias) of layer_norm: grad_x is the gradient of x and of the
    residual alike, with grad_sum (the gradient that reaches s by the residual path) added.
    grad_weight and grad_bias have one dtype, the weight's, or fp32 with
    weight_grad_dtype=torch.float32; grad_bias is None without want_bias.  out may be grad_y,
    sum or grad_sum itself."""
    gs = _matrix(grad_y, "grad_y")
    dev = grad_y.device
    dt = _dtype(grad_y, "grad_y")
    rows, width = grad_y.shape
    ss = _matrix(sum, "sum", grad_y.dtype, dev, rows, width)
    _vector(weight, "weight", (grad_y.dtype,), dev, width)
    _vector(mean, "mean", (torch.float32,), dev, rows)
    _vector(rstd, "rstd", (torch.float32,), dev, rows)
    ds = 0
    if grad_sum is not None:
        ds = _matrix(grad_sum, "grad_sum", grad_y.dtype, dev, rows, width)
    inputs = (weight, mean, rstd)
    if out is None:
        out = torch.empty(rows, width, dtype=grad_y.dtype, device=dev)
        os_ = width
    else:
        os_ = _matrix(out, "out", grad_y.dtype, dev, rows, width)
        _apart(out, "out", (grad_y, sum, grad_sum), inputs)
    given = weight_grad_out if weight_grad_out is not None else bias_grad_out if want_bias else None
    wdt = weight_grad_dtype or (given.dtype if given is not None else grad_y.dtype)
    if wdt not in (grad_y.dtype, torch.float32):
        raise ValueError(f"weight_grad_dtype: {wdt}, expected {grad_y.dtype} or torch.float32")
    if weight_grad_out is None:
        weight_grad_out = torch.empty(width, dtype=wdt, device=dev)
    else:
        _vector(weight_grad_out, "weight_grad_out", (wdt,), dev, width)
        _apart(weight_grad_out, "weight_grad_out", (), (*inputs, grad_y, sum, grad_sum, out))
    if not want_bias:
        if bias_grad_out is not None:
            raise ValueError("bias_grad_out: goes with want_bias")
    elif bias_grad_out is None:
        bias_grad_out = torch.empty(width, dtype=wdt, device=dev)
    else:
        _vector(bias_grad_out, "bias_grad_out", (wdt,), dev, width)
        _apart(bias_grad_out, "bias_grad_out", (),
               (*inputs, grad_y, sum, grad_sum, out, weight_grad_out))
    ws = _workspace(workspace, _layer_norm_backward_bytes(rows, width), dev)
    _run(dev, _layer_norm_backward, grad_y.data_ptr(), gs, sum.data_ptr(), ss, weight.data_ptr(),
         mean.data_ptr(), rstd.data_ptr(), grad_sum.data_ptr() if ds else None, ds, out.data_ptr(),
         os_, weight_grad_out.data_ptr(), bias_grad_out.data_ptr() if want_bias else None, rows,
         width, dt, _DTYPES[wdt], ws.data_ptr(), ws.numel())
    return out, weight_grad_out, bias_grad_out


# ---------------------------------------------------------------- 4-bit form


class Codes4(NamedTuple):
    """A matrix [rows, width] in the 4-bit form: codes [rows, 16 * G] (torch.float4_e2m1fn_x2, two
    elements a byte, the even one low; G = ceil(width / 32) groups, zeros behind the row's end)
    and scales [ceil(G / 16), rows, 4, 4] (torch.float8_e8m0fnu), that of a row's group n at
    [n // 16, row, n % 4, n // 4 % 4], as the matrix instructions take them; those of groups
    that do not exist are 1."""
    codes: torch.Tensor
    scales: torch.Tensor
    width: int


def _empty4(rows, width, device):
    groups = -(-width // 32)
    return (torch.empty(rows, 16 * groups, dtype=_FOUR, device=device),
            torch.empty(-(-groups // 16), rows, 4, 4, dtype=_SCALE, device=device))


def _codes4(c, name, device=None, width=None):
    """The rows of a matrix in the 4-bit form, which must lie as pack4 wrote it."""
    if not isinstance(c, Codes4):
        raise ValueError(f"{name}: {type(c).__name__}, expected Codes4")
    codes, scales, w = c
    if codes.dim() != 2 or not codes.is_cuda or (device is not None and codes.device != device):
        raise ValueError(f"{name}: codes of {codes.dim()} dimensions on {codes.device}, expected 2 "
                         f"on {device or 'a GPU'}")
    if width is not None and w != width:
        raise ValueError(f"{name}: width {w}, expected {width}")
    rows, groups = codes.shape[0], -(-w // 32)
    if codes.dtype != _FOUR or codes.shape[1] != 16 * groups or not codes.is_contiguous():
        raise ValueError(f"{name}: codes {codes.dtype} {tuple(codes.shape)}, expected {_FOUR} "
                         f"({rows}, {16 * groups}), contiguous")
    want = (-(-groups // 16), rows, 4, 4)
    if (scales.dtype != _SCALE or scales.device != codes.device or tuple(scales.shape) != want
            or not scales.is_contiguous()):
        raise ValueError(f"{name}: scales {scales.dtype} {tuple(scales.shape)} on {scales.device}, "
                         f"expected {_SCALE} {want} on {codes.device}, contiguous")
    return rows


def pack4(x, want="rows"):
    """A matrix in the 4-bit form: with want="rows" the Codes4 of x, with "columns" that of x.T
    (groups along x's columns), with "both" the two of them, from one pass over x."""
    xs = _matrix(x, "x")
    dev = x.device
    dt = _dtype(x, "x")
    if want not in ("rows", "columns", "both"):
        raise ValueError(f"want: {want!r}, expected one of ('rows', 'columns', 'both')")
    rows, width = x.shape
    a = b = None
    if want != "columns":
        a = Codes4(*_empty4(rows, width, dev), width)
    if want != "rows":
        b = Codes4(*_empty4(width, rows, dev), rows)
    if rows and width:
        _run(dev, _mx4_pack, x.data_ptr(), xs, a.codes.data_ptr() if a else None,
             a.scales.data_ptr() if a else None, b.codes.data_ptr() if b else None,
             b.scales.data_ptr() if b else None, rows, width, dt)
    return a if want == "rows" else b if want == "columns" else (a, b)


def unpack4(c, dtype, out=None):
    """The values of a matrix in the 4-bit form, each rounded once to dtype (exact in bf16 and
    fp32 but for 2^128, the form of magnitudes from 3.5 * 2^126 on: infinity)."""
    dt = _pick(_DTYPES, dtype, "dtype")
    rows = _codes4(c, "c")
    dev = c.codes.device
    if out is None:
        out = torch.empty(rows, c.width, dtype=dtype, device=dev)
        stride = c.width
    else:
        stride = _matrix(out, "out", dtype, dev, rows, c.width)
        _apart(out, "out", (), (c.codes, c.scales))
    if rows and c.width:
        _run(dev, _mx4_unpack, c.codes.data_ptr(), c.scales.data_ptr(), out.data_ptr(), stride, rows,
             c.width, dt)
    return out


def linear4(x, weight, dtype=None, out=None, workspace=None):
    """x @ weight.T for a weight in the 4-bit form (Codes4), summed in fp32 and rounded once to
    dtype.  x: a matrix, which is packed along its rows on the way (dtype: its own unless given;
    workspace= takes zs_mx4_linear_bytes), or Codes4 already (dtype: bf16 unless given).  With
    pack4's other orientations the same product gives the gradients: dx = linear4(dy, pack4(w,
    "columns")), dw = linear4(pack4(dy, "columns"), pack4(x, "columns"))."""
    packed = isinstance(x, Codes4)
    if packed:
        tokens, width = _codes4(x, "x"), x.width
        dev = x.codes.device
        inputs = (x.codes, x.scales)
    else:
        xs = _matrix(x, "x")
        tokens, width = x.shape
        dev = x.device
        xt = _dtype(x, "x")
        inputs = (x,)
    features = _codes4(weight, "weight", dev, width)
    if dtype is None:
        dtype = out.dtype if out is not None else torch.bfloat16 if packed else x.dtype
    dt = _pick(_DTYPES, dtype, "dtype")
    if out is None:
        out = torch.empty(tokens, features, dtype=dtype, device=dev)
        stride = features
    else:
        stride = _matrix(out, "out", dtype, dev, tokens, features)
        _apart(out, "out", (), (*inputs, weight.codes, weight.scales))
    if width == 0:
        return out.zero_()
    if packed:
        _run(dev, _mx4_product, x.codes.data_ptr(), x.scales.data_ptr(), weight.codes.data_ptr(),
             weight.scales.data_ptr(), out.data_ptr(), stride, tokens, features, width, dt)
    else:
        ws = _workspace(workspace, _mx4_linear_bytes(tokens, width), dev)
        _run(dev, _mx4_linear, x.data_ptr(), xs, weight.codes.data_ptr(), weight.scales.data_ptr(),
             out.data_ptr(), stride, tokens, features, width, xt, dt, ws.data_ptr(), ws.numel())
    return out


# ---------------------------------------------------------------- preference loss


class PreferenceOut(NamedTuple):
    """What preference_loss returns, for P pairs: loss [P], rewards [P, 2] (beta times the
    sequences' log ratios, the chosen one's first), margins [P] and lengths [P, 2] (the tokens
    that count, int32)."""
    loss: torch.Tensor
    rewards: torch.Tensor
    margins: torch.Tensor
    lengths: torch.Tensor


def _pairs(offsets, mask, device, tokens):
    if offsets.dim() != 1 or offsets.shape[0] % 2 == 0:
        raise ValueError(f"offsets: shape {tuple(offsets.shape)}, expected (2 * pairs + 1,)")
    _vector(offsets, "offsets", _ID_BYTES, device, offsets.shape[0])
    if mask is not None:
        _vector(mask, "mask", (torch.bool, torch.uint8), device, tokens)
    return offsets.shape[0] // 2


def preference_loss(loss, ref_loss, offsets, beta=0.1, kind="sigmoid", margin=0.0, smoothing=0.0,
                    average=False, mask=None, workspace=None):
    """The preference loss of pairs of packed sequences: loss and ref_loss (None: no reference)
    are the policy's and the reference's -log p of each token (linear_xent's), fp32 [tokens];
    sequence i is tokens offsets[i]:offsets[i + 1], pair p has 2p as the chosen and 2p + 1
    as the rejected one.  With each sequence's log ratio a = -sum(loss - ref_loss), or its
    mean over the tokens that count with average=True, m = beta * (a_chosen - a_rejected) -
    margin and the loss is -log sigma(m) ("sigmoid", with smoothing s (1 - s) times that and s
    times the same of -m), max(0, 1 - m) ("hinge") or (m - 1/2)^2 / beta^2 ("squared").  mask:
    True where a token counts; what loss and ref_loss hold elsewhere is not used."""
    tokens = loss.shape[0] if loss.dim() == 1 else -1
    dev = loss.device
    if not loss.is_cuda:
        raise ValueError(f"loss: on {dev}, expected a GPU")
    _vector(loss, "loss", (torch.float32,), dev, tokens)
    if ref_loss is not None:
        _vector(ref_loss, "ref_loss", (torch.float32,), dev, tokens)
    k = _pick(_KINDS, kind, "kind")
    pairs = _pairs(offsets, mask, dev, tokens)
    out, margins, rewards = loss.new_empty(pairs), loss.new_empty(pairs), loss.new_empty(pairs, 2)
    lengths = torch.empty(pairs, 2, dtype=torch.int32, device=dev)
    nbytes = _prefer_workspace_bytes(tokens, pairs)
    ws = _workspace(workspace, nbytes, dev) if nbytes != 256 else None  # 256: it is not used
    _run(dev, _prefer_forward, loss.data_ptr(), ref_loss.data_ptr() if ref_loss is not None else
         None, offsets.data_ptr(), mask.data_ptr() if mask is not None else None, out.data_ptr(),
         rewards.data_ptr(), margins.data_ptr(), lengths.data_ptr(), tokens, pairs, beta, margin,
         smoothing, k, int(average), _ID_BYTES[offsets.dtype], ws.data_ptr() if ws is not None else
         None, nbytes)
    return PreferenceOut(out, rewards, margins, lengths)


def preference_loss_backward(forward, offsets, grad_loss, tokens, beta=0.1, kind="sigmoid",
                             smoothing=0.0, average=False, mask=None, out=None):
    """The gradient of sum(grad_loss * preference_loss(...).loss) by each token's loss, fp32
    [tokens]: linear_xent_backward's grad_loss.  forward is what preference_loss returned for
    the same offsets, mask and settings, and the slope is the one at its margins, as they are held
    in fp32; tokens that do not count or lie in no sequence get 0."""
    dev = offsets.device
    if not offsets.is_cuda:
        raise ValueError(f"offsets: on {dev}, expected a GPU")
    if tokens < 0:
        raise ValueError(f"tokens: {tokens}, expected 0 or more")
    k = _pick(_KINDS, kind, "kind")
    pairs = _pairs(offsets, mask, dev, tokens)
    _vector(forward.margins, "margins", (torch.float32,), dev, pairs)
    lengths = forward.lengths
    if (tuple(lengths.shape) != (pairs, 2) or lengths.dtype != torch.int32 or lengths.device != dev
            or not lengths.is_contiguous()):
        raise ValueError(f"lengths: {lengths.dtype} {tuple(lengths.shape)} on {lengths.device}, "
                         f"expected torch.int32 ({pairs}, 2) on {dev}, contiguous")
    _vector(grad_loss, "grad_loss", (torch.float32,), dev, pairs)
    if out is None:
        out = torch.empty(tokens, dtype=torch.float32, device=dev)
    else:
        _vector(out, "out", (torch.float32,), dev, tokens)
        _apart(out, "out", (), (forward.margins, lengths, offsets, mask, grad_loss))
    _run(dev, _prefer_backward, forward.margins.data_ptr(), lengths.data_ptr(), offsets.data_ptr(),
         mask.data_ptr() if mask is not None else None, grad_loss.data_ptr(), out.data_ptr(),
         tokens, pairs, beta, smoothing, k, int(average), _ID_BYTES[offsets.dtype])
    return out


# ---------------------------------------------------------------- many gradients


def _grad_rows(g, o, i):
    """A gradient and its output as rows of adjacent elements: (rows, width, strides)."""
    for t, name in ((g, f"tensors[{i}]"), (o, f"out[{i}]")):
        if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1) or (
                t.stride(0) < t.shape[1] and t.shape[0] > 1):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, strides {t.stride()}: expected "
                             "contiguous, or a matrix (or its transpose) with adjacent elements "
                             "in a row")
    return (*g.shape, g.stride(0), o.stride(0))


class GradList:
    """Gradients of any types in many tensors, laid out once for grad_sumsq and clip_grads.

    tensors: contiguous ones, and matrices (or their transposes) with any row stride.  out: where
    their clipped values go, tensors of the same shapes and orientation in any of the types
    (views of a contribution buffer of ZeroShard); without it they are clipped in place.  The
    list holds its tensors and their addresses: a tensor must not be resized or given other
    memory.  Making it copies a table to the device and is not captured in a graph; the calls
    that use it are, and a graph reads the list's table at every replay: the list has to outlive
    it.  Calls on any stream hold the table's memory until their work is done; the tensors' is the
    caller's to hold, as for every call."""

    def __init__(self, tensors, out=None):
        self.tensors = list(tensors)
        self.out = list(out) if out is not None else None
        if not self.tensors:
            raise ValueError("tensors: an empty list")
        if self.out is not None and len(self.out) != len(self.tensors):
            raise ValueError(f"out: {len(self.out)} tensors, expected {len(self.tensors)}")
        self.device = self.tensors[0].device
        if not self.tensors[0].is_cuda:
            raise ValueError(f"tensors: on {self.device}, expected a GPU")
        with torch.cuda.device(self.device):
            if torch.cuda.is_current_stream_capturing():
                raise ValueError("a GradList copies its table to the device: it is made before a capture")
        dev, codes = self.device, {(a, b): _DTYPES[a] | _DTYPES[b] << 32 for a in _DTYPES for b in _DTYPES}
        records = []  # zs_grad_tensor, word by word
        for i, (g, o) in enumerate(zip(self.tensors, self.out or self.tensors)):
            code = codes.get((g.dtype, o.dtype))
            if code is None or g.device != dev or o.device != dev or o.shape != g.shape:
                raise ValueError(f"tensors[{i}]: {g.dtype} {tuple(g.shape)} on {g.device} to {o.dtype} "
                                 f"{tuple(o.shape)} on {o.device}, expected types of {tuple(_DTYPES)} "
                                 f"and one shape on {dev}")
            if g.is_contiguous() and o.is_contiguous():
                n = g.numel()
                records.append((g.data_ptr(), o.data_ptr(), 1, n, n, n, code))
                continue
            if g.dim() == 2 and not g.is_contiguous() and g.stride(0) == 1 and o.stride(0) == 1:
                g, o = g.t(), o.t()
            records.append((g.data_ptr(), o.data_ptr(), *_grad_rows(g, o, i), code))
        words = torch.tensor(records, dtype=torch.int64, device="cpu")
        self.pieces = int(_check(_grads_pieces(words.data_ptr(), len(records))))
        host = torch.empty(max(1, self.pieces) * 32, dtype=torch.uint8, device="cpu")
        _check(_grads_table(words.data_ptr(), len(records), host.data_ptr(), host.numel()))
        self.table = host.to(dev)
        self._streams = {_raw_stream(dev.index)}  # those that the table's memory is held for


def _grad_list(grads):
    if not isinstance(grads, GradList):
        return GradList(grads)
    stream = _raw_stream(grads.device.index)
    if stream not in grads._streams:
        grads.table.record_stream(torch.cuda.current_stream(grads.device))
        grads._streams.add(stream)
    return grads


def grad_sumsq(grads, out=None, workspace=None):
    """The sum of the squares of all elements of the tensors, a float64 scalar tensor (out=: one
    that is given).  grads: a GradList, or tensors.  Over several ranks it is summed by the
    caller before clip_grads."""
    grads = _grad_list(grads)
    dev = grads.device
    if out is None:
        out = torch.empty((), dtype=torch.float64, device=dev)
    elif out.dtype != torch.float64 or out.device != dev or out.numel() != 1:
        raise ValueError(f"out: {out.dtype} {tuple(out.shape)} on {out.device}, expected one "
                         f"torch.float64 on {dev}")
    ws = _workspace(workspace, _grads_workspace_bytes(grads.pieces), dev)
    _run(dev, _grads_sumsq, grads.table.data_ptr(), grads.pieces, out.data_ptr(), ws.data_ptr(),
         ws.numel())
    return out


def clip_grads(grads, max_norm, sumsq=None, workspace=None):
    """Writes min(1, max_norm / (norm + 1e-6)) times the gradients to their outputs (a GradList's
    out; in place otherwise) and returns their global norm, a float64 scalar tensor.  sumsq:
    grad_sumsq's result where it is summed over ranks; otherwise it is taken here."""
    grads = _grad_list(grads)
    dev = grads.device
    ws = None
    if sumsq is None:
        ws = _workspace(workspace, _grads_workspace_bytes(grads.pieces), dev)
    elif sumsq.dtype != torch.float64 or sumsq.device != dev or sumsq.numel() != 1:
        raise ValueError(f"sumsq: {sumsq.dtype} {tuple(sumsq.shape)} on {sumsq.device}, expected one "
                         f"torch.float64 on {dev}")
    norm = torch.empty((), dtype=torch.float64, device=dev)
    _run(dev, _grads_clip, grads.table.data_ptr(), grads.pieces, max_norm, sumsq.data_ptr() if sumsq
         is not None else None, norm.data_ptr(), ws.data_ptr() if ws is not None else None,
         ws.numel() if ws is not None else 0)
    return norm
