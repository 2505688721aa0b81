"""Host-only checks of the model operators' entry points: the library exports what
zeroshard_ops.h declares, every argument error is found before the device is
touched (there is none here), and the float64 formulas the GPU tests compare with
agree with differences of their own forward passes."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import _ops_ref as R
import sharded_optimizer_step_zero_amd as zs
from sharded_optimizer_step_zero_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an address no check dereferences


def test_library_exports_every_declared_operator():
    src = open(os.path.join(ROOT, "include", "zeroshard_ops.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(zs_[a-z0-9_]+)\s*\(", src)))
    lib = ctypes.CDLL(zs.LIB_PATH)
    for n in names:
        assert hasattr(lib, n) and callable(getattr(ops, n)), n
    assert sorted(ops.EXPORTED) == names


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "zeroshard_ops.h"\nint main(void) { return ZS_F32 + ZS_E4M3 + ZS_SILU; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only",
                    "-I", os.path.join(ROOT, "include"), str(src)], check=True)


def refused(call, *args):
    with pytest.raises(zs.ZeroShardError) as e:
        call(*args)
    assert e.value.code == zs.ZS_EINVAL
    return str(e.value)


def change(args, **at):
    """The argument list with some positions ("_3=...") replaced."""
    a = list(args)
    for k, v in at.items():
        a[int(k[1:])] = v
    return a


EMBED = [P, 64, P, P, 64, 10, 100, 64, 0, 1.0, 1, 8, 0]


@pytest.mark.parametrize("at, word", [
    (dict(_10=3), "type"), (dict(_10=-1), "type"), (dict(_11=2), "4 or 8"), (dict(_5=-1), "range"),
    (dict(_6=0), "range"), (dict(_6=(1 << 24) + 1), "range"), (dict(_7=0), "range"),
    (dict(_1=63), "stride"), (dict(_4=63), "stride"), (dict(_0=0), "NULL"), (dict(_2=0), "NULL"),
    (dict(_3=0), "NULL"), (dict(_0=P + 1), "aligned"), (dict(_2=P + 4), "aligned"),
    (dict(_9=float("nan")), "scale"), (dict(_9=float("inf")), "scale"),
    (dict(_5=1 << 31), "range")])
def test_embed_forward_refusals(at, word):
    assert word in refused(ops.zs_embed_forward, *change(EMBED, **at))


def embed_backward_args():
    n = ops.zs_embed_backward_bytes(10, 100, 64)
    assert n > 0 and n % 256 == 0
    return [P, 64, P, P, 64, 10, 100, 64, 0, 1.0, 1, 1, 8, 0, P, n, 0]


@pytest.mark.parametrize("at, word", [
    (dict(_10=7), "type"), (dict(_11=2), "gradient"), (dict(_12=3), "4 or 8"), (dict(_5=-1), "range"),
    (dict(_6=0), "range"), (dict(_7=0), "range"), (dict(_1=63), "stride"), (dict(_4=63), "stride"),
    (dict(_0=0), "NULL"), (dict(_3=0), "NULL"), (dict(_3=P + 1), "aligned"),
    (dict(_14=0), "workspace"), (dict(_14=P + 128), "workspace"), (dict(_15=255), "workspace"),
    (dict(_9=float("inf")), "scale")])
def test_embed_backward_refusals(at, word):
    assert word in refused(ops.zs_embed_backward, *change(embed_backward_args(), **at))


NORM = [P, 64, P, 64, P, P, 64, P, 64, P, P, P, 10, 64, 1e-6, 1, 0, 128, 0]


@pytest.mark.parametrize("at, word", [
    (dict(_15=9), "type"), (dict(_16=2), "8-bit"), (dict(_17=16), "8-bit"), (dict(_12=-1), "range"),
    (dict(_13=0), "range"), (dict(_13=65537), "range"), (dict(_14=-1.0), "eps"),
    (dict(_14=float("nan")), "eps"), (dict(_1=63), "stride"), (dict(_3=63), "stride"),
    (dict(_6=63), "stride"), (dict(_8=63), "stride"), (dict(_0=0), "NULL"), (dict(_4=0), "NULL"),
    (dict(_11=0), "NULL"), (dict(_2=0), "together"), (dict(_5=0), "together"),
    (dict(_9=0), "together"), (dict(_10=0), "together"), (dict(_0=P + 1), "aligned"),
    (dict(_11=P + 2), "aligned")])
def test_norm_forward_refusals(at, word):
    assert word in refused(ops.zs_norm_forward, *change(NORM, **at))


def norm_backward_args():
    n = ops.zs_norm_backward_bytes(10, 64)
    return [P, 64, P, 64, P, P, P, 64, P, 64, P, 10, 64, 1, 0, P, n, 0]


@pytest.mark.parametrize("at, word", [
    (dict(_13=5), "type"), (dict(_14=2), "weight"), (dict(_11=-1), "range"), (dict(_12=0), "range"),
    (dict(_1=63), "stride"), (dict(_3=63), "stride"), (dict(_7=63), "stride"),
    (dict(_9=63), "stride"), (dict(_0=0), "NULL"), (dict(_2=0), "NULL"), (dict(_4=0), "NULL"),
    (dict(_5=0), "NULL"), (dict(_8=0), "NULL"), (dict(_10=0), "NULL"), (dict(_10=P + 2), "aligned"),
    (dict(_15=0), "workspace"), (dict(_16=0), "workspace")])
def test_norm_backward_refusals(at, word):
    assert word in refused(ops.zs_norm_backward, *change(norm_backward_args(), **at))


PACK = [P, 64, P, P, 10, 64, 1, 0, 128, 0]
UNPACK = [P, P, P, 64, 10, 64, 1, 0, 128, 0]
GLU = [P, 128, P, 64, P, P, 10, 64, 1, 0, 0, 128, 0]
GLU_GRAD = [P, 64, P, P, P, 128, P, 64, 10, 64, 1, 0, 0, 128, 0]


@pytest.mark.parametrize("call, args, at, word", [
    (ops.zs_act8_pack, PACK, dict(_6=3), "type"), (ops.zs_act8_pack, PACK, dict(_7=2), "8-bit"),
    (ops.zs_act8_pack, PACK, dict(_8=100), "8-bit"), (ops.zs_act8_pack, PACK, dict(_4=-1), "range"),
    (ops.zs_act8_pack, PACK, dict(_5=0), "range"), (ops.zs_act8_pack, PACK, dict(_1=60), "stride"),
    (ops.zs_act8_pack, PACK, dict(_0=0), "NULL"), (ops.zs_act8_pack, PACK, dict(_2=0), "NULL"),
    (ops.zs_act8_pack, PACK, dict(_3=0), "NULL"), (ops.zs_act8_pack, PACK, dict(_0=P + 1), "aligned"),
    (ops.zs_act8_unpack, UNPACK, dict(_6=3), "type"), (ops.zs_act8_unpack, UNPACK, dict(_7=2), "8-bit"),
    (ops.zs_act8_unpack, UNPACK, dict(_3=63), "stride"), (ops.zs_act8_unpack, UNPACK, dict(_0=0), "NULL"),
    (ops.zs_act8_unpack, UNPACK, dict(_2=P + 1), "aligned"),
    (ops.zs_glu_forward, GLU, dict(_9=2), "activation"), (ops.zs_glu_forward, GLU, dict(_10=2), "8-bit"),
    (ops.zs_glu_forward, GLU, dict(_11=0), "8-bit"), (ops.zs_glu_forward, GLU, dict(_1=127), "stride"),
    (ops.zs_glu_forward, GLU, dict(_3=63), "stride"), (ops.zs_glu_forward, GLU, dict(_4=0), "together"),
    (ops.zs_glu_forward, GLU, dict(_0=0), "NULL"), (ops.zs_glu_forward, GLU, dict(_2=0), "NULL"),
    (ops.zs_glu_forward, GLU, dict(_7=0), "range"),
    (ops.zs_glu_backward, GLU_GRAD, dict(_11=2), "activation"),
    (ops.zs_glu_backward, GLU_GRAD, dict(_12=2), "8-bit"), (ops.zs_glu_backward, GLU_GRAD, dict(_13=8), "8-bit"),
    (ops.zs_glu_backward, GLU_GRAD, dict(_1=63), "stride"), (ops.zs_glu_backward, GLU_GRAD, dict(_5=64), "stride"),
    (ops.zs_glu_backward, GLU_GRAD, dict(_7=63), "stride"), (ops.zs_glu_backward, GLU_GRAD, dict(_0=0), "NULL"),
    (ops.zs_glu_backward, GLU_GRAD, dict(_2=0), "NULL"), (ops.zs_glu_backward, GLU_GRAD, dict(_4=0), "NULL"),
    (ops.zs_glu_backward, GLU_GRAD, dict(_6=P + 1), "aligned")])
def test_act8_refusals(call, args, at, word):
    assert word in refused(call, *change(args, **at))


def xent_args(backward):
    n = ops.zs_xent_workspace_bytes(P, 64, P, 64, 10, 100, 64, backward)
    assert n > 0 and n % 256 == 0
    if not backward:
        return [P, 64, P, 64, P, P, P, 10, 100, 64, 1, 8, P, n, 0]
    return [P, 64, P, 64, P, P, P, P, 64, P, 64, 10, 100, 64, 1, 8, P, n, 0]


@pytest.mark.parametrize("at, word", [
    (dict(_10=0), "bf16 or fp16"), (dict(_11=1), "4 or 8"), (dict(_7=-1), "range"), (dict(_8=0), "range"),
    (dict(_9=0), "range"), (dict(_9=65537), "range"), (dict(_1=63), "stride"), (dict(_3=63), "stride"),
    (dict(_1=(1 << 21) + 8), "stride"), (dict(_0=0), "NULL"), (dict(_2=0), "NULL"), (dict(_4=0), "NULL"),
    (dict(_5=0), "NULL"), (dict(_6=0), "NULL"), (dict(_4=P + 4), "aligned"), (dict(_0=P + 1), "aligned"),
    (dict(_12=0), "workspace"), (dict(_12=P + 64), "workspace"), (dict(_13=100), "workspace")])
def test_xent_forward_refusals(at, word):
    assert word in refused(ops.zs_xent_forward, *change(xent_args(0), **at))


@pytest.mark.parametrize("at, word", [
    (dict(_14=0), "bf16 or fp16"), (dict(_15=1), "4 or 8"), (dict(_11=-1), "range"), (dict(_12=0), "range"),
    (dict(_8=63), "stride"), (dict(_10=63), "stride"), (dict(_5=0), "NULL"), (dict(_6=0), "NULL"),
    (dict(_7=P + 1), "aligned"), (dict(_16=0), "workspace"), (dict(_17=100), "workspace"),
    (dict(_11=1 << 21), "many tokens")])
def test_xent_backward_refusals(at, word):
    assert word in refused(ops.zs_xent_backward, *change(xent_args(1), **at))


def test_sizes_of_zero_are_no_work():
    """No tokens: nothing to enqueue, so the calls succeed without a device."""
    ops.zs_embed_forward(*change(EMBED, _5=0, _2=0, _0=0, _3=0))
    ops.zs_norm_forward(*change(NORM, _12=0))
    ops.zs_act8_pack(*change(PACK, _4=0))
    ops.zs_act8_unpack(*change(UNPACK, _4=0))
    ops.zs_glu_forward(*change(GLU, _6=0))
    ops.zs_glu_backward(*change(GLU_GRAD, _8=0))
    ops.zs_xent_forward(*change(xent_args(0), _7=0))


def test_workspace_queries_out_of_range_are_zero():
    assert ops.zs_embed_backward_bytes(-1, 10, 10) == 0
    assert ops.zs_embed_backward_bytes(10, 0, 10) == 0
    assert ops.zs_norm_backward_bytes(10, 0) == 0
    assert ops.zs_xent_workspace_bytes(P, 64, P, 64, 10, 0, 64, 0) == 0
    # rows that cannot be read 16 bytes at a time need room for a copy
    assert ops.zs_xent_workspace_bytes(P, 65, P, 64, 10, 100, 65, 0) > \
        ops.zs_xent_workspace_bytes(P, 72, P, 72, 10, 100, 72, 0)
    assert ops.zs_xent_workspace_bytes(P + 2, 64, P, 64, 10, 100, 64, 0) > \
        ops.zs_xent_workspace_bytes(P, 64, P, 64, 10, 100, 64, 0)


def test_tensors_off_the_gpu_are_refused():
    x, w = torch.zeros(4, 64), torch.ones(64)
    h, i = x.bfloat16(), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: ops.embed(x, i), lambda: ops.embed_backward(x, i, 10), lambda: ops.norm(x, w),
                 lambda: ops.norm_backward(x, x, w, torch.ones(4)), lambda: ops.pack8(x),
                 lambda: ops.glu(x), lambda: ops.linear_xent(h, h, i),
                 lambda: ops.linear_xent_backward(h, h, i, torch.ones(4), torch.ones(4)),
                 lambda: ops.unpack8(x.to(torch.float8_e4m3fn), None, torch.float32),
                 lambda: ops.glu_backward(x, None, None)):
        with pytest.raises(ValueError, match="GPU"):
            call()


# ------------------------------------------------ the formulas against differences


def differs(f, x, grad, direction, h=1e-6):
    """(f(x + h d) - f(x - h d)) / 2h against <grad, d>: central differences of a
    float64 function of size ~1 are good to about 1e-9."""
    got = (f(x + h * direction) - f(x - h * direction)) / (2 * h)
    assert abs(float(got) - float((grad * direction).sum())) < 1e-7


def test_formulas_against_differences():
    g = torch.Generator().manual_seed(1)

    def r(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    x, w, dy, ds = r(5, 12), r(12), r(5, 12), r(5, 12)

    def norm_loss(x, w):
        return (R.norm(x, w, 1e-5)[0] * dy + x * ds).sum()
    dx, dw, _, _ = R.norm_grad(dy, x, w, R.norm(x, w, 1e-5)[1], ds)
    differs(lambda v: norm_loss(v, w), x, dx, r(5, 12))
    differs(lambda v: norm_loss(x, v), w, dw, r(12))

    for kind in ("silu", "gelu"):
        a, u_, do = r(7, 9), r(7, 9), r(7, 9)
        differs(lambda v: (R.act(v, kind)[0] * u_ * do).sum(), a, do * u_ * R.act(a, kind)[1], r(7, 9))

    ids = torch.tensor([3, 1, 3, -1, 0, 7, 3])
    table, dout = r(5, 4), r(7, 4)
    differs(lambda v: (R.embed(v, ids, 0.7) * dout).sum(), table, R.embed_grad(dout, ids, 5, 0.7)[0], r(5, 4))

    h, wt, gl = r(6, 8), r(11, 8), r(6)
    targets = torch.tensor([0, 10, -100, 4, 4, 11])
    _, _, _, _, _, dh, dwt, _, _, _ = R.xent(h, wt, targets, gl)
    differs(lambda v: (R.xent(v, wt, targets)[0] * gl).sum(), h, dh, r(6, 8))
    differs(lambda v: (R.xent(h, v, targets)[0] * gl).sum(), wt, dwt, r(11, 8))
