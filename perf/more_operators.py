"""The cases of the operators for training on preferences with products in 4 bits: what they
compute in plain form, and how a user calls them.

Four operators: the layer norm with its gradient, the microscaled 4-bit form with the
product of two packed matrices, the preference loss of pairs of packed sequences, and the
clipping of many tensors' gradients by their global norm into a contribution buffer.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# largest value, mantissa bits and least normal exponent of the narrow formats
CODES = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14), "e2m1": (6.0, 1, 0)}
EIGHT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def listed():
    return [
        # a layer's norm when the loss of a short text is evaluated
        dict(name="layer_norm_short", op="layer_norm", tokens=64, width=2048, dtype="bf16", code="none", group=32, keep=True),
        # a layer's norm in training on a wide model, its output going on in 8 bits only
        dict(name="layer_norm_train", op="layer_norm", tokens=16384, width=8192, dtype="bf16", code="e4m3", group=32, keep=False),
        # the backward pass of a layer's norm, with its weight's and its bias's gradient
        dict(name="layer_norm_grad", op="layer_norm_grad", tokens=32768, width=2048, dtype="bf16"),
        # the same on a ragged batch of a small model in fp16
        dict(name="layer_norm_grad_odd", op="layer_norm_grad", tokens=3001, width=1001, dtype="fp16"),
        # a weight of odd sizes put away in 4 bits for both of its products, and taken back
        dict(name="pack4_odd", op="pack4", tokens=517, width=2731, dtype="fp16"),
        # gate and up of a layer for 16 tokens: the weight is what is read
        dict(name="linear4_few", op="linear4", tokens=16, width=4096, features=22016, dtype="bf16"),
        # the same layer on one micro-batch: output, and the gradients of input and weight
        dict(name="linear4_train", op="linear4_grad", tokens=8192, width=4096, features=22016, dtype="bf16"),
        # a ragged batch on a small model whose sizes no tile divides
        dict(name="linear4_train_odd", op="linear4_grad", tokens=1003, width=1000, features=3125, dtype="bf16"),
        # four pairs of short answers: loss and gradient
        dict(name="preference_short", op="preference", pairs=4, tokens=1600, kind="sigmoid", beta=0.1, average=False, masked=True),
        # a batch of 256 pairs of long answers, lengths divided out, no reference model
        dict(name="preference_long", op="preference", pairs=256, tokens=1 << 20, kind="hinge", beta=2.0, average=True, masked=True),
        # the gradients of a GPT of 24 layers, vectors in fp32 and matrices in bf16, into a contribution
        dict(name="clip_gpt", op="clip", layers=24, width=2048, vocab=50304, dtype="mixed", out="bf16", max_norm=1.0),
        # ten thousand small tensors and a few matrices
        dict(name="clip_mixed", op="clip", tensors=10000, longest=4096, matrices=4, width=4096, dtype="bf16", out="bf16", max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_grad", "pack4", "linear4", "linear4_grad", "preference", "clip"])
    if op == "preference":
        pairs = _log(rng, 1, 512)
        average = rng.random() < 0.5
        return dict(op=op, pairs=pairs, tokens=max(2 * pairs, _log(rng, 64, 1 << 20)), kind=rng.choice(["sigmoid", "hinge", "squared"]),
                    beta=rng.choice([0.1, 0.5]) if not average else rng.choice([1.0, 2.0]), average=average, masked=average or rng.random() < 0.5)
    if op == "clip":
        dtype = rng.choice(["mixed", "bf16", "fp16", "fp32"])
        c = dict(op=op, dtype=dtype, out="fp16" if dtype == "fp16" else "bf16", max_norm=rng.choice([1.0, 0.1, 1e4]))
        if rng.random() < 0.5:
            w = _log(rng, 64, 2048)
            return dict(c, layers=_log(rng, 1, 24), width=w, vocab=min(_log(rng, 500, 50304), (1 << 26) // w))
        return dict(c, tensors=_log(rng, 1, 10000), longest=_log(rng, 16, 4096), matrices=rng.randrange(5), width=_log(rng, 64, 4096))
    t = _log(rng, 1, 16384)
    d = _log(rng, 64, 8192)
    if rng.random() < 0.5:  # widths of models are round; the others stay odd
        d = max(64, d // 64 * 64)
    c = dict(op=op, tokens=t, width=d, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "layer_norm":
        c.update(code=rng.choice(["none", "e4m3", "e5m2", "e2m1"]), keep=rng.random() < 0.5)
        c.update(group=32 if c["code"] == "e2m1" else rng.choice([32, 64, 128]))
    elif op.startswith("linear4"):
        n = _log(rng, 16, 28672)
        if rng.random() < 0.5:
            n = max(64, n // 64 * 64)
        c.update(features=n, tokens=max(1, min(t, 8192, 8192 * 4096 * 22016 // (n * d))))
    return c


def _shapes(case):
    """The tensors of a clip case: the same for every seed."""
    if "layers" in case:
        h = case["width"]
        one = [(h,), (h,), (3 * h, h), (h, h), (h,), (h,), (4 * h, h), (h, 4 * h)]
        return [(case["vocab"], h)] + one * case["layers"] + [(h,), (h,)]
    rng = random.Random(case["tensors"])
    got = [(rng.randint(1, case["longest"]),) for _ in range(case["tensors"])] + [(case["width"], case["width"])] * case["matrices"]
    rng.shuffle(got)
    return got


def _dtype_of(shape, dtype):
    return TYPES["fp32" if len(shape) == 1 else "bf16"] if dtype == "mixed" else TYPES[dtype]


def work(case):
    op = case["op"]
    if op == "preference":
        t = case["tokens"]
        return {"bytes": t * (4 + (0 if case["average"] else 4) + 4 + (1 if case["masked"] else 0)) + case["pairs"] * 40, "flops": 4 * t}
    if op == "clip":
        sizes = [(math.prod(s), _dtype_of(s, case["dtype"]).itemsize) for s in _shapes(case)]
        return {"bytes": sum(n * (e + TYPES[case["out"]].itemsize) for n, e in sizes), "flops": 3 * sum(n for n, _ in sizes)}
    t, d = case["tokens"], case["width"]
    e = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if op == "layer_norm":  # x, residual, weight, bias; the sum, statistics and what is wanted of the output
        code = {"none": 0, "e2m1": 0.5, "e4m3": 1, "e5m2": 1}[case["code"]] * t * d
        if code:
            code += t * -(-d // case["group"])
        if case["code"] == "e2m1":  # the values are taken back: codes read, 16 bits written
            code = 2 * code + 2 * t * d
        return {"bytes": 3 * t * d * e + 2 * d * e + 8 * t + code + (t * d * e if case["keep"] else 0), "flops": 8 * t * d}
    if op == "layer_norm_grad":  # dy, the sum, its gradient, the weight, statistics; dx, dw and db
        return {"bytes": 4 * t * d * e + d * e + 8 * t + 8 * d, "flops": 14 * t * d}
    if op == "pack4":  # put away both ways and taken back in 16 bits
        return {"bytes": t * d * e + 2 * (2 * t * d * 17 / 32) + 2 * t * d * 2, "flops": 6 * t * d}
    n = case["features"]
    w = n * d * 17 / 32
    if op == "linear4":
        return {"bytes": t * d * e + w + t * n * e, "flops": 2 * t * d * n}
    return {"bytes": 2 * t * d * e + 2 * w + 2 * t * n * e + n * d * e, "flops": 6 * t * d * n}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, s = case["op"], dict(case)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)

    def activations(*shape, dtype):
        # a few channels of an activation are far larger than the others, and some have an offset
        x = normal(*shape)
        big = uniform(shape[-1]) < 0.004
        return (x * torch.where(big, 24.0, 1.0) + torch.where(uniform(shape[-1]) < 0.02, 3.0, 0.0)).to(dtype)

    if op == "preference":
        n, t = 2 * case["pairs"], case["tokens"]
        # lengths over a factor of ten; what is left behind the last sequence is padding
        share = (0.1 + uniform(n)).double().cumsum(0)
        offsets = torch.zeros(n + 1, dtype=torch.int64, device=DEV)
        offsets[1:] = (share / share[-1] * int(t * 0.98)).long()
        loss = -torch.log(uniform(t).clamp(min=1e-6)) * 1.8
        s.update(loss=loss, ref_loss=None if case["average"] else loss + normal(t, std=0.1), offsets=offsets, mask=None)
        if case["masked"]:  # the prompt's tokens do not count; where they stand nothing was computed
            s["mask"] = uniform(t) < 0.8
            s["loss"] = torch.where(s["mask"], loss, torch.full_like(loss, math.nan))
        s.update(grad=torch.full((case["pairs"],), 1.0 / case["pairs"], device=DEV))
        return s
    if op == "clip":
        shapes = _shapes(case)
        total = sum(math.prod(x) for x in shapes)
        contribution = torch.zeros(total, dtype=TYPES[case["out"]], device=DEV)

        def gradients(n, dtype):
            # one in a hundred is far larger, one in twenty zero
            v = normal(n, std=1e-3)
            u = uniform(n)
            return torch.where(u < 0.05, torch.zeros_like(v), torch.where(u > 0.99, v * 100, v)).to(dtype)

        grads, views, at = [], [], 0
        pool = {}  # small tensors are cut from one buffer of random values
        small = {dt: sum(math.prod(x) + 8 for x in shapes if math.prod(x) <= 8192 and _dtype_of(x, case["dtype"]) == dt) for dt in TYPES.values()}
        for x in shapes:
            n, dt = math.prod(x), _dtype_of(x, case["dtype"])
            if n <= 8192:
                if dt not in pool:
                    pool[dt] = [gradients(small[dt], dt), 0]
                buffer, begin = pool[dt]
                grads.append(buffer[begin:begin + n].view(x))
                pool[dt][1] = begin + (n + 7) // 8 * 8
            else:
                grads.append(gradients(n, dt).view(x))
            views.append(contribution[at:at + n].view(x))
            at += n
        s.update(grads=grads, contribution=contribution)
        if own:  # the list of buffers is laid out once, like the step's plan
            from sharded_optimizer_step_zero_amd import ops
            s.update(list=ops.GradList(grads, out=views))
        return s
    t, d, dt = case["tokens"], case["width"], TYPES[case["dtype"]]
    if op == "layer_norm":
        s.update(x=normal(t, d, dtype=dt), residual=activations(t, d, dtype=dt), weight=(normal(d, std=0.1) + 1).to(dt), bias=normal(d, std=0.1, dtype=dt))
    elif op == "layer_norm_grad":
        x = activations(t, d, dtype=dt)
        mean = x.double().mean(1)
        rstd = (x.double().var(1, unbiased=False) + 1e-5).rsqrt()
        s.update(dy=normal(t, d, std=1e-2, dtype=dt), summed=x, mean=mean.float(), rstd=rstd.float(), dsum=normal(t, d, std=1e-2, dtype=dt), weight=(normal(d, std=0.1) + 1).to(dt))
    elif op == "pack4":
        s.update(x=activations(t, d, dtype=dt))
    else:
        n = case["features"]
        w = normal(n, d, std=1 / math.sqrt(d))
        s.update(x=activations(t, d, dtype=dt), weight=_packed(w))
        if op == "linear4_grad":  # gradients in fp16 carry a loss scale
            s.update(weight_t=_packed(w.t()), dy=normal(t, n, std=1.0 if dt == torch.float16 else 1e-3, dtype=dt))
    return s


# ------------------------------------------------------------------ plain forms


def _groups(x, group):
    """x's last axis in groups, zeros behind its end."""
    n = -(-x.shape[-1] // group)
    return torch.nn.functional.pad(x, (0, n * group - x.shape[-1])).view(*x.shape[:-1], n, group)


def _scaled(x, code, group):
    """x over its groups' scales, and the scales' exponents: the least that bring a group within the format."""
    p = _groups(x, group)
    amax = p.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e with m in [1/2, 1)
    top_m, top_e = math.frexp(CODES[code][0])
    e = e - top_e + (m > top_m)
    e = torch.where(amax == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    return p * torch.exp2(-e.to(x.dtype)).unsqueeze(-1), e


def _e8m0(e):
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _spans(e):
    """Sixteen neighbours of a row together, the n-th of them at [n % 4, n // 4]; those behind the end are zeros."""
    p = torch.nn.functional.pad(e, (0, -e.shape[1] % 16)).view(e.shape[0], -1, 4, 4)
    return p.permute(1, 0, 3, 2).contiguous()


def _four(v):
    """Rounded to the 4-bit format's values, ties to the even code."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(v.dtype)
    return torch.round(v / step) * step


def _packed(w):
    """(codes, scales, width) of a matrix in the 4-bit form: groups of 32, two codes a byte, the even element low."""
    v, e = _scaled(w.float(), "e2m1", 32)
    v = _four(v)
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    nibble = torch.bucketize(v.abs(), table) + torch.where(torch.signbit(v), 8, 0)
    nibble = nibble.to(torch.uint8).view(w.shape[0], -1, 2)
    return (nibble[..., 0] | nibble[..., 1] << 4).view(torch.float4_e2m1fn_x2), _e8m0(_spans(e)), w.shape[1]


def _values(packed):
    """The fp32 values of a packed matrix."""
    codes, scales, width = packed
    b = codes.view(torch.uint8)
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    table = torch.cat([table, -table])
    v = table[torch.stack([b & 15, b >> 4], -1).int()].view(b.shape[0], -1, 32)
    scales = torch.exp2(scales.view(torch.uint8).float() - 127).permute(1, 0, 3, 2).reshape(b.shape[0], -1)[:, :v.shape[1]]
    return (v * scales.unsqueeze(-1)).view(b.shape[0], -1)[:, :width]


def _quantised(x):
    """The fp32 values that a matrix has in the 4-bit form, along its rows, and the scales."""
    v, e = _scaled(x.float(), "e2m1", 32)
    back = (_four(v) * torch.exp2(e.float()).unsqueeze(-1)).view(x.shape[0], -1)[:, :x.shape[1]]
    return back, _e8m0(_spans(e))


def _plain(s):
    op = s["op"]
    if op == "preference":
        l = s["loss"].double() - (0 if s["ref_loss"] is None else s["ref_loss"].double())
        n = 2 * s["pairs"]
        place = torch.arange(s["tokens"], device=DEV)
        seq = torch.bucketize(place, s["offsets"], right=True) - 1
        counts = (seq >= 0) & (seq < n)
        if s["mask"] is not None:
            counts = counts & s["mask"]
        seq = torch.where(counts, seq, torch.full_like(seq, n))
        sums = torch.zeros(n + 1, dtype=torch.float64, device=DEV).index_add_(0, seq, torch.where(counts, l, torch.zeros_like(l)))
        length = torch.zeros(n + 1, dtype=torch.int64, device=DEV).index_add_(0, seq, counts.long())
        over = length.clamp(min=1).double() if s["average"] else torch.ones(n + 1, dtype=torch.float64, device=DEV)
        rewards = (-s["beta"] * sums / over)[:n].view(-1, 2)
        m = rewards[:, 0] - rewards[:, 1]
        if s["kind"] == "sigmoid":
            loss, slope = torch.log1p(torch.exp(-m.abs())) + torch.relu(-m), -1 / (1 + torch.exp(m))
        elif s["kind"] == "hinge":
            loss, slope = torch.relu(1 - m), torch.where(m < 1, -1.0, 0.0).double()
        else:
            loss, slope = ((m - 0.5) / s["beta"]).square(), 2 * (m - 0.5) / s["beta"] ** 2
        slope = slope * s["grad"]
        each = torch.zeros(n + 1, dtype=torch.float64, device=DEV)
        each[:n] = (torch.stack([-slope, slope], 1) * s["beta"]).view(-1) / over[:n]
        return dict(loss=loss.float(), rewards=rewards.float(), margins=m.float(), lengths=length[:n].view(-1, 2).int(), grad=each[seq].float())
    if op == "clip":
        flat = torch.cat([x.reshape(-1).float() for x in s["grads"]])
        norm = torch.sqrt(flat.double().square().sum())
        c = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
        s["contribution"].copy_(flat * c)
        return dict(contribution=s["contribution"], norm=norm)
    dt = TYPES[s["dtype"]]
    if op == "layer_norm":
        summed = (s["x"].float() + s["residual"].float()).to(dt)
        # a bit next to a border of the codes or of their scales decides: 64 bits where there are codes
        f = torch.float32 if s["code"] == "none" else torch.float64
        x = summed.to(f)
        mean = x.mean(1, keepdim=True)
        x = x - mean
        rstd = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-5)
        y = x * rstd * s["weight"].to(f) + s["bias"].to(f)
        out = dict(sum=summed, mean=mean[:, 0].float(), rstd=rstd[:, 0].float())
        if s["keep"]:
            out.update(y=y.to(dt))
        if s["code"] != "none":
            v, e = _scaled(y, s["code"], s["group"])
            out.update(scales=_e8m0(_spans(e) if s["code"] == "e2m1" else e))
            if s["code"] == "e2m1":
                back = _four(v) * torch.exp2(e.double()).unsqueeze(-1)
                out.update(values=back.view(s["tokens"], -1)[:, :s["width"]].to(torch.bfloat16))
            else:
                # to 8 bits in one rounding: what fp32 would cut off is kept in its last bit
                f = v.float()
                cut = f.double() != v
                bits = f.view(torch.int32)
                bits = torch.where(cut & (f.double().abs() > v.abs()), bits - 1, bits)
                f = torch.where(cut, bits | 1, bits).view(torch.float32)
                out.update(codes=f.view(s["tokens"], -1)[:, :s["width"]].to(EIGHT[s["code"]]))
        return out
    if op == "layer_norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        h = (s["summed"].float() - s["mean"][:, None]) * rstd
        g = dy * s["weight"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True)) + s["dsum"].float()
        return dict(dx=dx.to(dt), dw=(dy * h).sum(0), db=dy.sum(0))
    if op == "pack4":
        (a, ea), (b, eb) = _quantised(s["x"]), _quantised(s["x"].t())
        return dict(rows=a.to(torch.bfloat16), columns=b.to(torch.bfloat16), row_scales=ea, column_scales=eb)
    y = (_quantised(s["x"])[0] @ _values(s["weight"]).t()).to(dt)
    if op == "linear4":
        return y
    dx = (_quantised(s["dy"])[0] @ _values(s["weight_t"]).t()).to(dt)
    dw = (_quantised(s["dy"].t())[0] @ _quantised(s["x"].t())[0].t()).to(dt)
    return dict(y=y, dx=dx, dw=dw)


def _own(s):
    from sharded_optimizer_step_zero_amd import ops
    op = s["op"]
    if op == "preference":
        r = ops.preference_loss(s["loss"], s["ref_loss"], s["offsets"], beta=s["beta"], kind=s["kind"], average=s["average"], mask=s["mask"])
        grad = ops.preference_loss_backward(r, s["offsets"], s["grad"], s["tokens"], beta=s["beta"], kind=s["kind"], average=s["average"], mask=s["mask"])
        return dict(loss=r.loss, rewards=r.rewards, margins=r.margins, lengths=r.lengths, grad=grad)
    if op == "clip":
        norm = ops.clip_grads(s["list"], s["max_norm"])
        return dict(contribution=s["contribution"], norm=norm)
    dt = TYPES[s["dtype"]]
    if op == "layer_norm":
        code = None if s["code"] == "none" else s["code"]
        r = ops.layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=1e-5, code=code, group=s["group"], want_y=s["keep"])
        out = dict(sum=r.sum, mean=r.mean, rstd=r.rstd)
        if s["keep"]:
            out.update(y=r.y)
        if code == "e2m1":
            out.update(scales=r.scales, values=ops.unpack4(ops.Codes4(r.codes, r.scales, s["width"]), torch.bfloat16))
        elif code:
            out.update(scales=r.scales, codes=r.codes)
        return out
    if op == "layer_norm_grad":
        dx, dw, db = ops.layer_norm_backward(s["dy"], s["summed"], s["weight"], s["mean"], s["rstd"], grad_sum=s["dsum"], weight_grad_dtype=torch.float32)
        return dict(dx=dx, dw=dw, db=db)
    if op == "pack4":
        a, b = ops.pack4(s["x"], want="both")
        return dict(rows=ops.unpack4(a, torch.bfloat16), columns=ops.unpack4(b, torch.bfloat16), row_scales=a.scales, column_scales=b.scales)
    if op == "linear4":
        return ops.linear4(s["x"], ops.Codes4(*s["weight"]))
    x, x_t = ops.pack4(s["x"], want="both")
    dy, dy_t = ops.pack4(s["dy"], want="both")
    return dict(y=ops.linear4(x, ops.Codes4(*s["weight"]), dtype=dt), dx=ops.linear4(dy, ops.Codes4(*s["weight_t"]), dtype=dt), dw=ops.linear4(dy_t, x_t, dtype=dt))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits


def _exact_pack(y, code, group):
    """(values of the codes, scales) in fp64, the scale the least power of two that holds the group."""
    top, bits, low = CODES[code]
    rows, d = y.shape
    n = (d + group - 1) // group
    full = torch.zeros(rows, n * group, dtype=torch.float64, device=y.device)
    full[:, :d] = y
    largest = full.view(rows, n, group).abs().max(2).values
    need = torch.ceil(torch.log2((largest / top).clamp(min=2.0 ** -127)))
    # log2 may land on either side of a whole number
    need = torch.where(top * torch.exp2(need - 1) >= largest, need - 1, need)
    need = torch.where(top * torch.exp2(need) < largest, need + 1, need)
    scale = torch.exp2(need.clamp(-127, 127))
    v = full / scale.repeat_interleave(group, 1)
    place = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** (low - 1)))).clamp(min=low)
    step = torch.exp2(place - bits)
    return (torch.round(v / step) * step)[:, :d], scale


def _exact_values(x):
    codes, scale = _exact_pack(x.double(), "e2m1", 32)
    return codes * scale.repeat_interleave(32, 1)[:, :x.shape[1]], _exact_spans(scale)


def _exact_spans(scale):
    """Scales in the order in which the 4-bit form holds them."""
    rows, n = scale.shape
    out = torch.ones(-(-n // 16), rows, 4, 4, dtype=torch.float64, device=DEV)
    for g in range(n):
        out[g // 16, :, g % 4, g // 4 % 4] = scale[:, g]
    return out


def _exact_unpacked(packed):
    codes, scales, width = packed
    b = codes.view(torch.uint8).long()
    out = torch.empty(b.shape[0], 2 * b.shape[1], dtype=torch.float64, device=DEV)
    for at, nibble in ((0, b % 16), (1, b // 16)):
        low, high = nibble % 2, nibble // 2 % 4
        size = torch.where(high == 0, low * 0.5, (1 + 0.5 * low) * torch.exp2(high.double() - 1))
        out[:, at::2] = torch.where(nibble >= 8, -size, size)
    power = torch.exp2(scales.view(torch.uint8).double() - 127)
    for g in range(-(-width // 32)):
        out[:, 32 * g:32 * g + 32] *= power[g // 16, :, g % 4, g // 4 % 4, None]
    return out[:, :width]


def _times(a, b):
    """a b^T in pieces of rows."""
    b = b.t().contiguous()
    return torch.cat([torch.mm(p, b) for p in a.split(2048)])


def exact(case, seed):
    s = prepare(case, seed)
    op, f = case["op"], torch.float64
    if op == "preference":
        edges = s["offsets"].tolist()
        n, t = 2 * case["pairs"], case["tokens"]
        counted = torch.ones(t, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"]
        diff = s["loss"].to(f) if s["ref_loss"] is None else s["loss"].to(f) - s["ref_loss"].to(f)
        a, length = torch.zeros(n, dtype=f, device=DEV), torch.zeros(n, dtype=torch.int64, device=DEV)
        for i in range(n):
            part = diff[edges[i]:edges[i + 1]][counted[edges[i]:edges[i + 1]]]
            length[i] = part.numel()
            a[i] = -part.sum() / (max(1, part.numel()) if case["average"] else 1)
        a = (a * case["beta"]).view(-1, 2).requires_grad_()
        m = a[:, 0] - a[:, 1]
        if case["kind"] == "sigmoid":
            loss = torch.nn.functional.softplus(-m)
        elif case["kind"] == "hinge":
            loss = (1 - m).clamp(min=0)
        else:
            loss = (m / case["beta"] - 1 / (2 * case["beta"])) ** 2
        da, = torch.autograd.grad((loss * s["grad"].to(f)).sum(), a)
        grad = torch.zeros(t, dtype=f, device=DEV)
        for i, v in enumerate(da.reshape(-1).tolist()):
            c = counted[edges[i]:edges[i + 1]]
            over = max(1, int(length[i])) if case["average"] else 1
            grad[edges[i]:edges[i + 1]] = torch.where(c, -case["beta"] * v / over, 0.0)
        return dict(loss=loss.detach(), rewards=a.detach(), margins=m.detach(), lengths=None, grad=grad)
    if op == "clip":
        norm = math.sqrt(math.fsum(torch.stack([torch.linalg.vector_norm(x, dtype=f) ** 2 for x in s["grads"]]).tolist()))
        c = min(1.0, case["max_norm"] / (norm + 1e-6))
        return dict(contribution=torch.cat([x.reshape(-1).to(f).mul_(c) for x in s["grads"]]), norm=torch.tensor(norm, dtype=f))
    t, d = case["tokens"], case["width"]
    if op == "layer_norm":
        total = s["x"].to(f) + s["residual"].to(f)
        held = total.to(TYPES[case["dtype"]]).to(f)  # the operator normalises the sum that it stores
        var, mean = torch.var_mean(held, 1, correction=0)
        r = (var + 1e-5).pow(-0.5)
        y = (held - mean[:, None]) * r[:, None] * s["weight"].to(f) + s["bias"].to(f)
        out = dict(sum=total, mean=mean, rstd=r)
        if case["keep"]:
            out.update(y=y)
        if case["code"] != "none":
            codes, scale = _exact_pack(y, case["code"], case["group"])
            out.update(scales=_exact_spans(scale) if case["code"] == "e2m1" else scale)
            if case["code"] == "e2m1":
                out.update(values=codes * scale.repeat_interleave(32, 1)[:, :d])
            else:
                out.update(codes=codes)
        return out
    if op == "layer_norm_grad":
        r, dy = s["rstd"].to(f)[:, None], s["dy"].to(f)
        h = (s["summed"].to(f) - s["mean"].to(f)[:, None]) * r
        g = dy * s["weight"].to(f)
        inner = (g.sum(1, keepdim=True) + h * (g * h).sum(1, keepdim=True)) / d
        return dict(dx=(g - inner) * r + s["dsum"].to(f), dw=(dy * h).sum(0), db=dy.sum(0))
    if op == "pack4":
        (a, ea), (b, eb) = _exact_values(s["x"]), _exact_values(s["x"].t())
        return dict(rows=a, columns=b, row_scales=ea, column_scales=eb)
    x, w = _exact_values(s["x"])[0], _exact_unpacked(s["weight"])
    y = _times(x, w)
    if op == "linear4":
        return y
    dy, w_t = _exact_values(s["dy"])[0], _exact_unpacked(s["weight_t"])
    dy_t, x_t = _exact_values(s["dy"].t())[0], _exact_values(s["x"].t())[0]
    return dict(y=y, dx=_times(dy, w_t), dw=_times(dy_t, x_t))
