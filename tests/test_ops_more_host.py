"""Host-only checks of the layer norm, the 4-bit form, the preference loss and the clipping of many
gradients: argument errors are found before the device is touched, tables of gradients are
laid out and checked on the host, and the float64 formulas that the GPU tests compare
with agree with differences of their own forward passes."""
import ctypes
import struct

import pytest
import torch

import _more_ref as M
from sharded_optimizer_step_zero_amd import ops
from test_ops_host import P, change, refused

INF = float("inf")
NAN = float("nan")


LAYER_NORM = [P, 64, P, 64, P, P, P, 64, P, 64, P, P, P, P, 10, 64, 1e-5, 1, 0, 128, 0]


@pytest.mark.parametrize("at, word", [
    (dict(_17=3), "type"), (dict(_18=3), "8-bit"), (dict(_18=-1), "8-bit"), (dict(_19=16), "8-bit"),
    (dict(_18=2), "groups of 32"), (dict(_18=2, _19=64), "groups of 32"), (dict(_14=-1), "range"),
    (dict(_14=1 << 31), "range"), (dict(_15=0), "range"), (dict(_15=65537), "range"),
    (dict(_16=-1.0), "eps"), (dict(_16=NAN), "eps"), (dict(_16=INF), "eps"), (dict(_1=63), "stride"),
    (dict(_3=63), "stride"), (dict(_7=63), "stride"), (dict(_9=63), "stride"), (dict(_0=0), "NULL"),
    (dict(_4=0), "NULL"), (dict(_12=0), "NULL"), (dict(_13=0), "NULL"), (dict(_2=0), "together"),
    (dict(_6=0), "together"), (dict(_10=0), "together"), (dict(_11=0), "together"),
    (dict(_0=P + 1), "aligned"), (dict(_5=P + 1), "aligned"), (dict(_12=P + 2), "aligned"),
    (dict(_18=2, _19=32, _10=P + 2), "aligned"), (dict(_14=(1 << 31) - 1), "too many")])
def test_layer_norm_forward_refusals(at, word):
    assert word in refused(ops.zs_layer_norm_forward, *change(LAYER_NORM, **at))


def layer_norm_backward_args(width=64):
    n = ops.zs_layer_norm_backward_bytes(10, width)
    assert n > 0 and n % 256 == 0
    return [P, width, P, width, P, P, P, P, width, P, width, P, P, 10, width, 1, 0, P, n, 0]


@pytest.mark.parametrize("at, word", [
    (dict(_15=3), "type"), (dict(_16=2), "weight"), (dict(_13=-1), "range"), (dict(_14=0), "range"),
    (dict(_14=65537), "range"), (dict(_1=63), "stride"), (dict(_3=63), "stride"),
    (dict(_8=63), "stride"), (dict(_10=63), "stride"), (dict(_0=0), "NULL"), (dict(_2=0), "NULL"),
    (dict(_4=0), "NULL"), (dict(_5=0), "NULL"), (dict(_6=0), "NULL"), (dict(_9=0), "NULL"),
    (dict(_11=0), "NULL"), (dict(_11=P + 2), "aligned"), (dict(_12=P + 2), "aligned"),
    (dict(_5=P + 2), "aligned"), (dict(_17=0), "workspace"), (dict(_17=P + 128), "workspace"),
    (dict(_18=255), "workspace")])
def test_layer_norm_backward_refusals(at, word):
    assert word in refused(ops.zs_layer_norm_backward, *change(layer_norm_backward_args(), **at))


def test_layer_norm_backward_of_too_many_wide_rows():
    a = layer_norm_backward_args(8200)
    assert "too many rows" in refused(ops.zs_layer_norm_backward, *change(a, _13=1 << 22))
    assert ops.zs_layer_norm_backward_bytes(-1, 64) == 0
    assert ops.zs_layer_norm_backward_bytes(1, 65537) == 0


PACK4 = [P, 64, P, P, P, P, 10, 64, 1, 0]
UNPACK4 = [P, P, P, 64, 10, 64, 1, 0]
PRODUCT = [P, P, P, P, P, 70, 10, 70, 64, 1, 0]
LINEAR = [P, 64, P, P, P, 70, 10, 70, 64, 1, 1, P, 1 << 20, 0]


@pytest.mark.parametrize("call, args, at, word", [
    (ops.zs_mx4_pack, PACK4, dict(_8=3), "type"), (ops.zs_mx4_pack, PACK4, dict(_6=-1), "range"),
    (ops.zs_mx4_pack, PACK4, dict(_6=(1 << 24) + 1), "range"), (ops.zs_mx4_pack, PACK4, dict(_7=0), "range"),
    (ops.zs_mx4_pack, PACK4, dict(_6=(1 << 20) + 1), "along them"),
    (ops.zs_mx4_pack, PACK4, dict(_1=63), "stride"), (ops.zs_mx4_pack, PACK4, dict(_0=0), "NULL"),
    (ops.zs_mx4_pack, PACK4, dict(_2=0), "together"), (ops.zs_mx4_pack, PACK4, dict(_5=0), "together"),
    (ops.zs_mx4_pack, PACK4, dict(_2=0, _3=0, _4=0, _5=0), "NULL"),
    (ops.zs_mx4_pack, PACK4, dict(_2=P + 8), "aligned"), (ops.zs_mx4_pack, PACK4, dict(_5=P + 4), "aligned"),
    (ops.zs_mx4_pack, PACK4, dict(_0=P + 1), "aligned"),
    (ops.zs_mx4_pack, PACK4, dict(_1=1 << 20, _6=1 << 20, _7=1 << 20), "too many"),
    (ops.zs_mx4_pack, PACK4, dict(_1=1 << 20, _4=0, _5=0, _6=1 << 24, _7=1 << 20), "too many"),
    (ops.zs_mx4_unpack, UNPACK4, dict(_6=-1), "type"), (ops.zs_mx4_unpack, UNPACK4, dict(_5=0), "range"),
    (ops.zs_mx4_unpack, UNPACK4, dict(_3=63), "stride"), (ops.zs_mx4_unpack, UNPACK4, dict(_1=0), "NULL"),
    (ops.zs_mx4_unpack, UNPACK4, dict(_2=P + 1), "aligned"), (ops.zs_mx4_unpack, UNPACK4, dict(_0=P + 8), "aligned"),
    (ops.zs_mx4_product, PRODUCT, dict(_9=3), "type"), (ops.zs_mx4_product, PRODUCT, dict(_8=0), "range"),
    (ops.zs_mx4_product, PRODUCT, dict(_8=(1 << 20) + 1), "range"),
    (ops.zs_mx4_product, PRODUCT, dict(_6=-1), "range"), (ops.zs_mx4_product, PRODUCT, dict(_7=-1), "range"),
    (ops.zs_mx4_product, PRODUCT, dict(_5=69), "stride"), (ops.zs_mx4_product, PRODUCT, dict(_4=0), "NULL"),
    (ops.zs_mx4_product, PRODUCT, dict(_1=0), "NULL"), (ops.zs_mx4_product, PRODUCT, dict(_3=P + 8), "aligned"),
    (ops.zs_mx4_product, PRODUCT, dict(_4=P + 1), "aligned"),
    (ops.zs_mx4_product, PRODUCT, dict(_5=1 << 24, _6=1 << 24, _7=1 << 24), "too many"),
    (ops.zs_mx4_linear, LINEAR, dict(_6=-1), "range"), (ops.zs_mx4_linear, LINEAR, dict(_8=0), "range"),
    (ops.zs_mx4_linear, LINEAR, dict(_1=63), "stride"), (ops.zs_mx4_linear, LINEAR, dict(_5=69), "stride"),
    (ops.zs_mx4_linear, LINEAR, dict(_0=0), "NULL"), (ops.zs_mx4_linear, LINEAR, dict(_2=0), "NULL"),
    (ops.zs_mx4_linear, LINEAR, dict(_4=0), "NULL"), (ops.zs_mx4_linear, LINEAR, dict(_9=5), "type"),
    (ops.zs_mx4_linear, LINEAR, dict(_10=5), "type"), (ops.zs_mx4_linear, LINEAR, dict(_11=0), "workspace"),
    (ops.zs_mx4_linear, LINEAR, dict(_11=P + 16), "workspace"), (ops.zs_mx4_linear, LINEAR, dict(_12=500), "workspace"),
    (ops.zs_mx4_linear, LINEAR, dict(_3=P + 8), "aligned"), (ops.zs_mx4_linear, LINEAR, dict(_0=P + 1), "aligned")])
def test_mx4_refusals(call, args, at, word):
    assert word in refused(call, *change(args, **at))


def prefer_args():
    n = ops.zs_prefer_workspace_bytes(1 << 20, 1)
    assert n > ops.zs_prefer_workspace_bytes(100, 1) > 0
    return [P, P, P, P, P, P, P, P, 1 << 20, 1, 0.1, 0.0, 0.0, 0, 0, 8, P, n, 0]


@pytest.mark.parametrize("at, word", [
    (dict(_8=-1), "range"), (dict(_8=1 << 31), "range"), (dict(_9=-1), "range"),
    (dict(_9=(1 << 22) + 1), "range"), (dict(_15=2), "4 or 8"), (dict(_13=3), "kind"),
    (dict(_10=0.0), "beta"), (dict(_10=NAN), "beta"), (dict(_10=INF), "beta"),
    (dict(_11=INF), "margin"), (dict(_12=-0.1), "smoothing"), (dict(_12=0.6), "smoothing"),
    (dict(_12=0.1, _13=1), "smoothing"), (dict(_2=0), "offsets"), (dict(_2=P + 4), "offsets"),
    (dict(_0=0), "NULL"), (dict(_4=0), "NULL"), (dict(_7=0), "NULL"), (dict(_0=P + 2), "aligned"),
    (dict(_16=0), "workspace"), (dict(_16=P + 8), "workspace"), (dict(_17=256), "workspace")])
def test_prefer_forward_refusals(at, word):
    assert word in refused(ops.zs_prefer_forward, *change(prefer_args(), **at))


PREFER_GRAD = [P, P, P, P, P, P, 100, 4, 0.1, 0.0, 0, 0, 8, 0]


@pytest.mark.parametrize("at, word", [
    (dict(_6=-1), "range"), (dict(_7=-1), "range"), (dict(_8=-1.0), "beta"), (dict(_9=0.7), "smoothing"),
    (dict(_10=7), "kind"), (dict(_12=1), "4 or 8"), (dict(_2=0), "offsets"), (dict(_0=0), "NULL"),
    (dict(_1=0), "NULL"), (dict(_4=0), "NULL"), (dict(_5=0), "NULL"), (dict(_5=P + 1), "aligned")])
def test_prefer_backward_refusals(at, word):
    assert word in refused(ops.zs_prefer_backward, *change(PREFER_GRAD, **at))


# ---------------------------------------------------------------- tables of gradients

PIECE = 4096


def record(grad, out, rows, width, gs=None, os_=None, dt=1, ot=1):
    return ops.GradTensor(grad, out, rows, width, gs or width, os_ or width, dt, ot)


@pytest.mark.parametrize("r, word", [
    (record(P, P, 1, 8, dt=3), "type"), (record(P, P, 1, 8, ot=-1), "type"),
    (record(P, P, -1, 8), "range"), (record(P, P, 1, -8), "range"),
    (record(P, P, 1 << 30, 1 << 30), "range"), (record(P, P, 2, 8, gs=7), "stride"),
    (record(P, P, 2, 8, os_=7), "stride"), (record(0, P, 1, 8), "NULL"),
    (record(P + 1, P, 1, 8), "aligned"), (record(P, P + 2, 1, 8, ot=0), "aligned"),
    (record(P, P, 1 << 27, 8, gs=16), "too many")])
def test_grads_list_refusals(r, word):
    assert word in refused(ops.zs_grads_pieces, [r])


def test_a_list_of_too_many_rows_is_refused_without_counting_them():
    assert "too many" in refused(ops.zs_grads_pieces, [record(P, P, 1 << 40, 1, gs=2)])
    assert "too many" in refused(ops.zs_grads_pieces, [record(P, P, 1 << 26, 1, gs=2), record(P, P, 1, 1)])
    assert ops.zs_grads_pieces([record(P, P, 1 << 26, 1, gs=2)]) == 1 << 26
    assert ops.zs_grads_pieces([record(P, P, 1 << 40, 0, gs=2)]) == 0


def table(records):
    n = ops.zs_grads_pieces(records)
    buf = ctypes.create_string_buffer(max(1, n) * 32)
    ops.zs_grads_table(records, ctypes.addressof(buf), n * 32)
    return [struct.unpack_from("<QQiiii", buf.raw, 32 * i) for i in range(n)]


def test_grads_table():
    big = 2 * PIECE + 5
    got = table([record(P, 2 * P, 1, big, dt=0, ot=1), record(8 * P, 0, 3, 10, gs=16, dt=2),
                 record(16 * P, 16 * P, 0, 8), record(32 * P, 32 * P, 4, 6, dt=1)])
    # whole pieces come first
    assert got == [(P, 2 * P, PIECE, 0, 1, 0), (P + 4 * PIECE, 2 * P + 2 * PIECE, PIECE, 0, 1, 0),
                   (P + 8 * PIECE, 2 * P + 4 * PIECE, 5, 0, 1, 0), (8 * P, 0, 10, 2, 2, 0),
                   (8 * P + 32, 0, 10, 2, 2, 0), (8 * P + 64, 0, 10, 2, 2, 0),
                   (32 * P, 32 * P, 24, 1, 1, 0)]
    got = table([record(P, 2 * P, 1, 7), record(8 * P, 0, 1, PIECE)])
    assert got == [(8 * P, 0, PIECE, 1, 1, 0), (P, 2 * P, 7, 1, 1, 0)]
    assert table([]) == []
    assert "small" in refused(ops.zs_grads_table, [record(P, P, 1, 8)], P, 31)
    assert "table" in refused(ops.zs_grads_table, [record(P, P, 1, 8)], 0, 32)


@pytest.mark.parametrize("records, bad", [
    ([record(P, P, 1, 8), record(P, 2 * P, 1, 8)], True),                  # read by one, written by another
    ([record(P, P, 1, 8), record(P, P, 1, 8)], True),                      # the same tensor twice, in place
    ([record(P, 2 * P, 1, 8), record(P, 4 * P, 1, 8)], False),             # read twice
    ([record(P, 2 * P, 1, 8), record(4 * P, 2 * P + 14, 1, 8)], True),     # outputs share an element
    ([record(P, 2 * P, 1, 8), record(4 * P, 2 * P + 16, 1, 8)], False),
    ([record(P, P, 1, 8, dt=0, ot=1)], True),                              # in place, another type
    ([record(P, P + 2, 1, 8)], True),
    ([record(P, P + 32, 3, 8, gs=32, os_=32)], False),                     # side by side in one matrix
    ([record(P, P + 14, 3, 8, gs=32, os_=32)], True),
    ([record(P, 0, 1, 8), record(P, 0, 1, 8)], False)])                    # nothing written
def test_grads_outputs_that_overlap(records, bad):
    if bad:
        n = ops.zs_grads_pieces(records)
        buf = ctypes.create_string_buffer(n * 32)
        assert "overlaps" in refused(ops.zs_grads_table, records, ctypes.addressof(buf), n * 32)
    else:
        table(records)


@pytest.mark.parametrize("call, args, word", [
    (ops.zs_grads_sumsq, [P, -1, P, P, 1 << 20, 0], "range"), (ops.zs_grads_sumsq, [0, 1, P, P, 1 << 20, 0], "NULL"),
    (ops.zs_grads_sumsq, [P, 1, 0, P, 1 << 20, 0], "NULL"), (ops.zs_grads_sumsq, [P, 1, P + 4, P, 1 << 20, 0], "aligned"),
    (ops.zs_grads_sumsq, [P + 8, 1, P, P, 1 << 20, 0], "aligned"), (ops.zs_grads_sumsq, [P, 1, P, 0, 1 << 20, 0], "workspace"),
    (ops.zs_grads_sumsq, [P, 1, P, P, 255, 0], "workspace"),(ops.zs_grads_clip, [P, 1, 0.0, P, P, 0, 0, 0], "max_norm"), (ops.zs_grads_clip, [P, 1, NAN, P, P, 0, 0, 0], "max_norm"),
    (ops.zs_grads_clip, [P, 1, INF, P, P, 0, 0, 0], "max_norm"), (ops.zs_grads_clip, [0, 1, 1.0, P, P, 0, 0, 0], "NULL"),
    (ops.zs_grads_clip, [P, 1, 1.0, 0, P, 0, 0, 0], "workspace"), (ops.zs_grads_clip, [P, 1, 1.0, 0, P, P, 255, 0], "workspace"),
    (ops.zs_grads_clip, [P, 1, 1.0, 0, P, P + 8, 1 << 20, 0], "workspace"), (ops.zs_grads_clip, [P, 1, 1.0, P, P + 4, 0, 0, 0], "aligned"),
    (ops.zs_grads_clip, [P, 1, 1.0, P + 4, P, 0, 0, 0], "aligned"), (ops.zs_grads_clip, [P, -1, 1.0, P, P, 0, 0, 0], "range")])
def test_grads_refusals(call, args, word):
    assert word in refused(call, *args)


# ---------------------------------------------------------------- tensors


def test_tensors_off_the_gpu_are_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    v = torch.zeros(64, dtype=torch.bfloat16)
    f = torch.zeros(4)
    o = torch.zeros(3, dtype=torch.int64)
    c = ops.Codes4(torch.zeros(4, 32, dtype=torch.uint8).view(torch.float4_e2m1fn_x2),
                   torch.zeros(1, 4, 4, 4, dtype=torch.uint8).view(torch.float8_e8m0fnu), 64)
    for call in (lambda: ops.layer_norm(x, v), lambda: ops.layer_norm_backward(x, x, v, f, f),
                 lambda: ops.pack4(x), lambda: ops.unpack4(c, torch.float32), lambda: ops.linear4(x, c),
                 lambda: ops.linear4(c, c), lambda: ops.preference_loss(f, None, o),
                 lambda: ops.preference_loss_backward(None, o, f, 4), lambda: ops.GradList([x]),
                 lambda: ops.clip_grads([x], 1.0)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="empty"):
        ops.GradList([])


# ---------------------------------------------------------------- formulas


def slope(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_layer_norm_gradient_is_the_difference_of_the_layer_norm():
    g = torch.Generator().manual_seed(0)
    s = torch.randn(5, 12, generator=g).double() + 2
    w, b, dy = (torch.randn(12, generator=g).double(), torch.randn(12, generator=g).double(),
                torch.randn(5, 12, generator=g).double())
    _, mean, rstd, _ = M.layer_norm(s, w, b, 1e-5)
    dx, dw, db, *_ = M.layer_norm_grad(dy, s, w, mean, rstd)
    for v, d, f in ((s, dx, lambda q: (M.layer_norm(q, w, b, 1e-5)[0] * dy).sum()),
                    (w, dw, lambda q: (M.layer_norm(s, q, b, 1e-5)[0] * dy).sum()),
                    (b, db, lambda q: (M.layer_norm(s, w, q, 1e-5)[0] * dy).sum())):
        along = torch.randn(v.shape, generator=g).double()
        # differences over 2e-6: off by a part in 1e9 of values of about 10
        assert abs(float(slope(f, v, along) - (d * along).sum())) < 1e-6


@pytest.mark.parametrize("kind, smoothing", [("sigmoid", 0.0), ("sigmoid", 0.1), ("hinge", 0.0), ("squared", 0.0)])
@pytest.mark.parametrize("average", [False, True])
def test_preference_gradient_is_the_difference_of_the_loss(kind, smoothing, average):
    g = torch.Generator().manual_seed(1)
    loss = torch.randn(40, generator=g).double()
    ref, grad = torch.randn(40, generator=g).double(), torch.rand(3, generator=g).double()
    mask = torch.rand(40, generator=g) < 0.8
    o = [2, 9, 9, 20, 26, 27, 38]
    f = lambda q: (M.prefer(q, ref, o, mask, 0.3, kind, 0.2, smoothing, average)[0] * grad).sum()  # noqa: E731
    d = M.prefer(loss, ref, o, mask, 0.3, kind, 0.2, smoothing, average, grad)[6]
    along = torch.randn(40, generator=g).double()
    assert abs(float(slope(f, loss, along) - (d * along).sum())) < 1e-6


def test_four_bit_values_by_hand():
    v, b = M.pack4(torch.tensor([[6.0, 5.0, 2.5, 1.75, 1.25, 0.75, 0.25, -0.26]]).double())
    assert v[0, 0, :8].tolist() == [6, 4, 2, 2, 1, 1, 0, -0.5] and b.tolist() == [[127]]
    v, b = M.pack4(torch.tensor([[6.001, -3.0, 0.0]]).double())
    assert v[0, 0, :3].tolist() == [3, -1.5, 0] and b.tolist() == [[128]]
    assert M.pack4(torch.tensor([[1.0, float("inf")]]).double())[1].tolist() == [[255]]
    assert M.pack4(torch.zeros(1, 3).double())[1].tolist() == [[0]]
