"""The gated unit far out on both sides, in fp32."""
import pytest
import torch

import _ops_ref as R
from sharded_optimizer_step_zero_amd import ops

from test_gpu_ops_embed import DEV

pytestmark = pytest.mark.gpu


def test_silu_keeps_its_digits():
    """e^-|x| is held to a few units whatever x, down to fp32's subnormals: the exponential,
    the sum, the quotient and two products, two units each at most."""
    x = torch.cat([torch.linspace(-110, 110, 40001), torch.linspace(-2, 2, 4000), torch.tensor([0.0, -0.0, 1e-30, -1e-30])])
    n = x.numel()
    gate_up = torch.cat([x, torch.ones(n)])[None].to(DEV)
    out = ops.glu(gate_up, act="silu", code=None)[0]
    want = (x.double() / (1 + torch.exp(-x.double())))[None]
    R.close(out, want, want.abs() * 16 * R.E + 2 * R.sub(torch.float32), "silu")


def test_silu_gradient_keeps_its_digits():
    """The same of the derivative, from the values that the checkpoint holds; its two parts
    cancel near -1.28."""
    x = torch.linspace(-105, 105, 8192)
    gate_up = torch.cat([x, torch.full((8192,), 1.0)])[None].to(DEV)
    _, codes, scales = ops.glu(gate_up, act="silu", group=32)
    dgu, again = ops.glu_backward(torch.ones(1, 8192, device=DEV), codes, scales, group=32, want_out=True)
    g = R.unpack(codes[:, :8192], R.byte_of(scales)[:, 0], 32)
    f, slope, _, size = R.act(g, "silu")
    R.close(dgu[:, :8192], slope, size * 24 * R.E + 4 * R.sub(torch.float32) * (1 + g.abs()), "slope")
    R.close(dgu[:, 8192:], f, f.abs() * 16 * R.E + 2 * R.sub(torch.float32), "act")
    R.close(again, f, f.abs() * 16 * R.E + 2 * R.sub(torch.float32), "out")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinite_gates(act, dtype):
    """As the formula has it: infinity at infinity, and no value at -infinity."""
    x = torch.tensor([[float("inf"), float("-inf"), float("nan"), -3e38, 3e38, -300.0, -256.0, 1, 1, 1, 1, 1, 1, 1]],
                     dtype=dtype, device=DEV)
    out = ops.glu(x, act=act, code=None)[0][0].cpu()
    assert out[0] == float("inf") and torch.isnan(out[1:3]).all()
    assert out[3] == 0 and out[4] == x[0, 4].cpu() and not out[5:].any()
