"""The language-model operators' cases: what they compute in plain form, and how a user calls them.

Four operators make the gradient contributions that the shard step reads: the
token embedding, the root-mean-square norm with the residual's addition and an
8-bit output, the gated unit whose checkpoint is held in 8 bits (with the packing
alone), and the loss of a linear head over a large vocabulary.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# exponent of the largest value's leading bit (the largest value is 1.75 times that),
# mantissa bits and least normal exponent of the 8-bit formats
CODES = {"e4m3": (torch.float8_e4m3fn, 8, 3, -6), "e5m2": (torch.float8_e5m2, 15, 2, -14)}


def listed():
    return [
        # the next token of 32 sequences enters the model
        dict(name="embed_decode", op="embed", tokens=32, vocab=50304, width=2048, dtype="bf16", scale=45.25),
        # one micro-batch of 16k tokens: the table's gradient contribution
        dict(name="embed_grad", op="embed_grad", tokens=16384, vocab=32000, width=4096, dtype="bf16", scale=64.0),
        # a short, ragged batch on a small model in fp16
        dict(name="embed_grad_odd", op="embed_grad", tokens=3001, vocab=32003, width=1001, dtype="fp16", scale=1.0),
        # a layer's norm while 32 sequences decode
        dict(name="norm_decode", op="norm", tokens=32, width=4096, dtype="bf16", code="e4m3", group=128, keep=True),
        # a layer's norm in training, its output going on in 8 bits only
        dict(name="norm_train", op="norm", tokens=16384, width=8192, dtype="bf16", code="e4m3", group=128, keep=False),
        # the backward pass of a layer's norm
        dict(name="norm_grad", op="norm_grad", tokens=8192, width=4096, dtype="bf16"),
        # the gated unit of a layer in training, keeping its input in 8 bits
        dict(name="glu_train", op="glu", tokens=8192, width=11008, dtype="bf16", act="silu", code="e4m3", group=128),
        # its backward pass from those 8 bits on a wide model
        dict(name="glu_grad", op="glu_grad", tokens=4096, width=28672, dtype="bf16", act="silu", code="e4m3", group=128),
        # an activation of odd width put away and taken back
        dict(name="pack_odd", op="pack", tokens=517, width=2731, dtype="fp16", code="e5m2", group=64),
        # the loss of 64 tokens when a model is evaluated
        dict(name="xent_eval", op="xent", tokens=64, vocab=50304, width=2048, dtype="bf16"),
        # the loss and the gradients of one micro-batch
        dict(name="xent_train", op="xent_grad", tokens=8192, vocab=32000, width=4096, dtype="bf16"),
        # a ragged batch on a small model whose sizes no tile divides
        dict(name="xent_train_odd", op="xent_grad", tokens=1003, vocab=32003, width=1000, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "glu", "glu_grad", "pack", "xent", "xent_grad"])
    t = _log(rng, 1, 16384)
    d = _log(rng, 64, 8192)
    if rng.random() < 0.5:  # widths of models are round; the others stay odd
        d = max(64, d // 64 * 64)
    c = dict(op=op, tokens=t, width=d, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op.startswith("embed"):
        c.update(vocab=_log(rng, 500, 65536), scale=rng.choice([1.0, 0.5, round(math.sqrt(d), 2)]))
        c["vocab"] = min(c["vocab"], (1 << 28) // d)
    elif op.startswith("xent"):
        c.update(vocab=_log(rng, 500, 65536), dtype=rng.choice(["bf16", "bf16", "fp16"]))
        c["width"] = d = min(d, 4096)
        c["tokens"] = max(1, min(t, 8192, 8192 * 4096 * 32000 // (c["vocab"] * d), (1 << 28) // c["vocab"]))
    elif op == "norm":
        c.update(code=rng.choice(["e4m3", "e4m3", "e5m2"]), group=rng.choice([32, 64, 128]), keep=rng.random() < 0.5)
    elif op.startswith("glu"):
        c["width"] = min(c["width"] * 3 + rng.randrange(3), 28672)
        c["tokens"] = max(1, min(t, 4096 * 28672 // c["width"]))
        c.update(act=rng.choice(["silu", "gelu"]), code=rng.choice(["e4m3", "e4m3", "e5m2"]), group=rng.choice([32, 64, 128]))
    elif op == "pack":
        c.update(code=rng.choice(["e4m3", "e5m2"]), group=rng.choice([32, 64, 128]))
    return c


def work(case):
    t, d = case["tokens"], case["width"]
    e = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    v, g = case.get("vocab", 0), case.get("group", 1)
    groups = -(-d // g)
    op = case["op"]
    if op == "embed":
        return {"bytes": t * 8 + 2 * t * d * e, "flops": t * d}
    if op == "embed_grad":
        return {"bytes": t * 8 + t * d * e + v * d * e, "flops": 2 * t * d}
    if op == "norm":  # x, residual, weight; the sum, rstd, codes, scales and the 16-bit output where it is kept
        return {"bytes": 3 * t * d * e + d * e + 4 * t + t * d + t * groups + (t * d * e if case["keep"] else 0), "flops": 6 * t * d}
    if op == "norm_grad":  # dy, the sum, its gradient, the weight, rstd; dx and dw
        return {"bytes": 4 * t * d * e + d * e + 4 * t + 4 * d, "flops": 10 * t * d}
    if op == "glu":
        return {"bytes": 3 * t * d * e + 2 * t * d + 2 * t * groups, "flops": 8 * t * d}
    if op == "glu_grad":  # dout, codes, scales; the input's gradient and the output again
        return {"bytes": 4 * t * d * e + 2 * t * d + 2 * t * groups, "flops": 16 * t * d}
    if op == "pack":  # put away and taken back: the codes are written and read
        return {"bytes": 2 * t * d * e + 2 * (t * d + t * groups), "flops": 4 * t * d}
    if op == "xent":
        return {"bytes": (t + v) * d * e + 16 * t, "flops": 2 * t * v * d}
    return {"bytes": 2 * (t + v) * d * e + 20 * t, "flops": 6 * t * v * d}


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def prepare(case, seed):
    g = _generator(seed)
    t, d, dt = case["tokens"], case["width"], TYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)

    def tokens(n, vocab, skipped):
        # frequencies of a language: an id's probability falls as one over its rank
        u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
        ids = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp_(0, vocab - 1)
        if skipped:  # one token in 50 is padding
            ids = torch.where(torch.rand(n, generator=g, device=DEV) < 0.02, torch.full_like(ids, -100), ids)
        return ids

    def activations(*shape):
        # a few channels of an activation are far larger than the others
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
        big = torch.rand(shape[-1], generator=g, device=DEV) < 0.004
        return (x * torch.where(big, 24.0, 1.0)).to(dt)

    s = dict(case)
    if op == "embed":
        s.update(table=normal(case["vocab"], d, std=0.02), ids=tokens(t, case["vocab"], False))
    elif op == "embed_grad":
        s.update(dout=normal(t, d, std=1e-2), ids=tokens(t, case["vocab"], True))
    elif op == "norm":
        s.update(x=normal(t, d), residual=activations(t, d), weight=normal(d, std=0.1, dtype=torch.float32).add_(1).to(dt))
    elif op == "norm_grad":
        x = activations(t, d)
        rstd = (x.float().square().mean(-1) + 1e-6).rsqrt()
        s.update(dy=normal(t, d, std=1e-2), summed=x, rstd=rstd, dsum=normal(t, d, std=1e-2), weight=normal(d, std=0.1, dtype=torch.float32).add_(1).to(dt))
    elif op == "glu":
        s.update(gate_up=activations(t, 2 * d))
    elif op == "glu_grad":
        codes, scales = _pack(activations(t, 2 * d).float().view(t, 2, d), case["code"], case["group"])
        s.update(dout=normal(t, d, std=1e-2), codes=codes.reshape(t, 2 * d), scales=scales)
    elif op == "pack":
        s.update(x=activations(t, d))
    else:
        targets = tokens(t, case["vocab"], True)
        s.update(hidden=normal(t, d), weight=normal(case["vocab"], d, std=2.0 / math.sqrt(d)), targets=targets)
        if op == "xent_grad":  # the mean over the tokens that count
            n = (targets >= 0).sum().clamp(min=1).float()
            # gradients in fp16 carry a loss scale, here one that keeps them in range
            s.update(gloss=(4096.0 if case["dtype"] == "fp16" else 1.0) / n * torch.ones(t, device=DEV))
    return s


# ------------------------------------------------------------------ plain forms


def _pack(x, code, group):
    """Codes and power-of-two scales of x's last axis in fp32, group by group."""
    dtype, top, _, _ = CODES[code]
    d = x.shape[-1]
    n = -(-d // group)
    p = torch.nn.functional.pad(x, (0, n * group - d)).view(*x.shape[:-1], n, group)
    amax = p.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e with m in [1/2, 1)
    e = e - 1 + (m > 0.875) - top
    e = torch.where(amax == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    fine = torch.isfinite(amax)
    scaled = torch.where(fine.unsqueeze(-1), torch.ldexp(p, -e.unsqueeze(-1)), torch.zeros_like(p))
    codes = scaled.view(*x.shape[:-1], n * group)[..., :d].to(dtype)
    byte = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return codes, byte.view(torch.float8_e8m0fnu)


def _unpack(codes, scales, group):
    d = codes.shape[-1]
    s = torch.ldexp(torch.ones((), device=codes.device), scales.view(torch.uint8).int() - 127)
    s = torch.where(scales.view(torch.uint8) == 255, torch.full_like(s, math.nan), s)
    return codes.float() * s.repeat_interleave(group, -1)[..., :d]


def _act(x, kind):
    """The activation and its derivative."""
    if kind == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1 + th), 0.5 * (1 + th) + 0.5 * x * (1 - th * th) * c * (1 + 3 * 0.044715 * x * x)


def _plain(s):
    op, dt = s["op"], TYPES[s["dtype"]]
    if op == "embed":
        return (s["table"][s["ids"]].float() * s["scale"]).to(dt)
    if op == "embed_grad":
        keep = ((s["ids"] >= 0) & (s["ids"] < s["vocab"])).nonzero().squeeze(1)
        total = torch.zeros(s["vocab"], s["width"], device=DEV)
        total.index_add_(0, s["ids"][keep], s["dout"][keep].float())
        return (total * s["scale"]).to(dt)
    if op == "norm":
        summed = (s["x"].float() + s["residual"].float()).to(dt)
        x = summed.float()
        rstd = 1 / torch.sqrt((x * x).mean(-1) + 1e-6)
        y = x * rstd[:, None] * s["weight"].float()
        codes, scales = _pack(y, s["code"], s["group"])
        out = dict(sum=summed, rstd=rstd, codes=codes, scales=scales)
        return dict(out, y=y.to(dt)) if s["keep"] else out
    if op == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = s["summed"].float() * rstd
        wdy = dy * s["weight"].float()
        dx = rstd * (wdy - xhat * (wdy * xhat).mean(-1, keepdim=True)) + s["dsum"].float()
        return dict(dx=dx.to(dt), dw=(dy * xhat).sum(0))
    if op == "glu":
        x = s["gate_up"].float().view(s["tokens"], 2, s["width"])
        codes, scales = _pack(x, s["code"], s["group"])
        return dict(out=(_act(x[:, 0], s["act"])[0] * x[:, 1]).to(dt), codes=codes.reshape(s["tokens"], -1), scales=scales)
    if op == "glu_grad":
        x = _unpack(s["codes"].view(s["tokens"], 2, s["width"]), s["scales"], s["group"])
        f, df = _act(x[:, 0], s["act"])
        do, u = s["dout"].float(), x[:, 1]
        return dict(dgate_up=torch.cat([do * u * df, do * f], 1).to(dt), out=(f * u).to(dt))
    if op == "pack":
        codes, scales = _pack(s["x"].float(), s["code"], s["group"])
        return dict(codes=codes, scales=scales, back=_unpack(codes, scales, s["group"]).to(dt))
    h, w = s["hidden"].float(), s["weight"].float()
    logits = h @ w.t()
    counts = (s["targets"] >= 0) & (s["targets"] < s["vocab"])
    at = torch.where(counts, s["targets"], torch.zeros_like(s["targets"]))[:, None]
    top = logits.amax(1, keepdim=True)
    lse = torch.log(torch.exp(logits - top).sum(1)) + top[:, 0]
    loss = torch.where(counts, lse - logits.gather(1, at)[:, 0], torch.zeros_like(lse))
    if op == "xent":
        return dict(loss=loss, lse=lse)
    grad = torch.exp(logits - lse[:, None])
    grad.scatter_add_(1, at, -torch.ones_like(lse)[:, None])
    grad *= torch.where(counts, s["gloss"], torch.zeros_like(lse))[:, None]
    return dict(loss=loss, lse=lse, dhidden=(grad @ w).to(dt), dweight=(grad.t() @ h).to(dt))


def _own(s):
    from sharded_optimizer_step_zero_amd import ops
    op = s["op"]
    if op == "embed":
        return ops.embed(s["table"], s["ids"], scale=s["scale"])
    if op == "embed_grad":
        return ops.embed_backward(s["dout"], s["ids"], s["vocab"], scale=s["scale"])
    if op == "norm":
        r = ops.norm(s["x"], s["weight"], residual=s["residual"], eps=1e-6, code=s["code"], group=s["group"], want_y=s["keep"])
        out = dict(sum=r.sum, rstd=r.rstd, codes=r.codes, scales=r.scales)
        return dict(out, y=r.y) if s["keep"] else out
    if op == "norm_grad":
        dx, dw = ops.norm_backward(s["dy"], s["summed"], s["weight"], s["rstd"], grad_sum=s["dsum"], weight_grad_dtype=torch.float32)
        return dict(dx=dx, dw=dw)
    if op == "glu":
        out, codes, scales = ops.glu(s["gate_up"], act=s["act"], code=s["code"], group=s["group"])
        return dict(out=out, codes=codes, scales=scales)
    if op == "glu_grad":
        dgu, out = ops.glu_backward(s["dout"], s["codes"], s["scales"], act=s["act"], group=s["group"], want_out=True)
        return dict(dgate_up=dgu, out=out)
    if op == "pack":
        codes, scales = ops.pack8(s["x"], code=s["code"], group=s["group"])
        return dict(codes=codes, scales=scales, back=ops.unpack8(codes, scales, s["x"].dtype, group=s["group"]))
    loss, lse = ops.linear_xent(s["hidden"], s["weight"], s["targets"])
    if op == "xent":
        return dict(loss=loss, lse=lse)
    dh, dw = ops.linear_xent_backward(s["hidden"], s["weight"], s["targets"], lse, s["gloss"])
    return dict(loss=loss, lse=lse, dhidden=dh, dweight=dw)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits


def _grid64(x, code):
    """x rounded to the nearest value of the 8-bit format, ties to even, in fp64 (|x| within its range)."""
    _, _, bits, low = CODES[code]
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** (low - 1)))).clamp(min=low)
    step = torch.exp2(e - bits)
    return torch.round(x / step) * step


def _exact_pack(y, code, group):
    """(values of the codes, scales) with the scale the least power of two that holds the group."""
    top = CODES[code][1]
    rows, d = y.shape
    n = (d + group - 1) // group
    full = torch.zeros(rows, n * group, dtype=torch.float64, device=y.device)
    full[:, :d] = y
    full = full.view(rows, n, group)
    largest = full.abs().max(2).values
    need = torch.ceil(torch.log2((largest / (1.75 * 2.0 ** top)).clamp(min=2.0 ** -127)))
    # log2 may land on either side of a whole number
    need = torch.where(1.75 * 2.0 ** top * torch.exp2(need - 1) >= largest, need - 1, need)
    need = torch.where(1.75 * 2.0 ** top * torch.exp2(need) < largest, need + 1, need)
    scale = torch.exp2(need.clamp(-127, 127))
    codes = _grid64(full / scale[:, :, None], code).view(rows, n * group)[:, :d]
    return codes, scale


def _spread(scale, group, d):
    return scale[:, torch.arange(d, device=scale.device) // group]


def _act64(x, kind):
    if kind == "silu":
        q = 1 / (1 + torch.exp(-x))
        return x * q, q + x * q * (1 - q)
    k = (2 / math.pi) ** 0.5
    z = k * (x + 0.044715 * x ** 3)
    q = 1 / (1 + torch.exp(-2 * z))  # (1 + tanh z) / 2
    return x * q, q + x * 2 * q * (1 - q) * k * (1 + 0.134145 * x ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op, t, d = case["op"], case["tokens"], case["width"]
    f = torch.float64
    if op == "embed":
        return torch.index_select(s["table"], 0, s["ids"]).to(f).mul_(case["scale"])
    if op == "embed_grad":
        # sums of sorted tokens as differences would lose digits: one column block at a time
        good = (s["ids"] >= 0) & (s["ids"] < case["vocab"])
        out = torch.zeros(case["vocab"], d, dtype=f, device=DEV)
        rows = s["ids"][good]
        for a in range(0, d, 1024):
            part = s["dout"][good][:, a:a + 1024].to(f) * case["scale"]
            out[:, a:a + 1024].scatter_add_(0, rows[:, None].expand(-1, part.shape[1]), part)
        return out
    if op == "norm":
        total = s["x"].to(f) + s["residual"].to(f)
        held = total.to(TYPES[case["dtype"]]).to(f)  # the operator normalises the sum that it stores
        r = (held.pow(2).sum(1) / d + 1e-6).pow(-0.5)
        y = held * s["weight"].to(f) * r[:, None]
        codes, scales = _exact_pack(y, case["code"], case["group"])
        out = dict(sum=total, rstd=r, codes=codes, scales=scales)
        return dict(out, y=y) if case["keep"] else out
    if op == "norm_grad":
        r = s["rstd"].to(f)[:, None]
        dy, x, w = s["dy"].to(f), s["summed"].to(f), s["weight"].to(f)
        inner = (dy * w * x).sum(1, keepdim=True) * r ** 3 / d
        return dict(dx=dy * w * r - x * inner + s["dsum"].to(f), dw=(dy * x * r).sum(0))
    if op == "glu":
        gate, up = s["gate_up"][:, :d].to(f), s["gate_up"][:, d:].to(f)
        pairs = [_exact_pack(v, case["code"], case["group"]) for v in (gate, up)]
        return dict(out=_act64(gate, case["act"])[0] * up, codes=torch.cat([p[0] for p in pairs], 1), scales=torch.stack([p[1] for p in pairs], 1))
    if op == "glu_grad":
        power = torch.exp2(s["scales"].view(torch.uint8).to(f) - 127)
        gate = s["codes"][:, :d].to(f) * _spread(power[:, 0], case["group"], d)
        up = s["codes"][:, d:].to(f) * _spread(power[:, 1], case["group"], d)
        a, slope = _act64(gate, case["act"])
        do = s["dout"].to(f)
        return dict(dgate_up=torch.cat([do * slope * up, do * a], 1), out=a * up)
    if op == "pack":
        codes, scales = _exact_pack(s["x"].to(f), case["code"], case["group"])
        return dict(codes=codes, scales=scales, back=codes * _spread(scales, case["group"], d))
    w = s["weight"].to(f)
    target = s["targets"]
    live = (target >= 0) & (target < case["vocab"])
    loss = torch.zeros(t, dtype=f, device=DEV)
    lse = torch.zeros(t, dtype=f, device=DEV)
    dh = torch.zeros(t, d, dtype=f, device=DEV)
    dw = torch.zeros(case["vocab"], d, dtype=f, device=DEV)
    for a in range(0, t, 2048):  # tokens are independent; the weight's gradient adds up
        b = min(t, a + 2048)
        h = s["hidden"][a:b].to(f)
        z = torch.mm(h, w.t().contiguous())
        lse[a:b] = torch.logsumexp(z, 1)
        row = torch.arange(b - a, device=DEV)[live[a:b]]
        col = target[a:b][live[a:b]]
        loss[a:b][live[a:b]] = lse[a:b][live[a:b]] - z[row, col]
        if op == "xent_grad":
            z = torch.exp(z - lse[a:b, None])
            z[row, col] -= 1
            z = z * torch.where(live[a:b], s["gloss"][a:b].to(f), torch.zeros(b - a, dtype=f, device=DEV))[:, None]
            dh[a:b] = torch.mm(z, w)
            dw += torch.mm(z.t().contiguous(), h)
    return dict(loss=loss, lse=lse) if op == "xent" else dict(loss=loss, lse=lse, dhidden=dh, dweight=dw)
