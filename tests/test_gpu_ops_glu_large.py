"""The gated unit's gradient where grad_out times up passes fp32 and the product with the
slope does not."""
import pytest
import torch

from sharded_optimizer_step_zero_amd import ops

from test_gpu_ops_embed import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_infinity_on_the_way(act, dtype):
    x = torch.empty(1, 256, dtype=dtype, device=DEV)
    x[:, :32], x[:, 32:64], x[:, 64:96], x[:, 96:128] = -1000.0, -30.0, -1e30, 0.0
    x[:, 128:] = 2.0 ** 125
    _, codes, scales = ops.glu(x, act=act, group=32)
    for size in (1.0, 16.0, -2.0 ** 100):
        dgu, _ = ops.glu_backward(torch.full((1, 128), size, dtype=dtype, device=DEV), codes, scales, act=act, group=32)
        dgate = dgu[:, :96].double()
        assert not torch.isnan(dgu[:, :96]).any()
        assert not dgate[:, :32].any() and not dgate[:, 64:].any()  # the slope there is 0
    # 16 * 2^125 is past fp32; times a slope of -30 e^-30 it is 1.9e27
    dgu, _ = ops.glu_backward(torch.full((1, 128), 16.0, dtype=dtype, device=DEV), codes, scales, act=act, group=32)
    assert torch.isfinite(dgu[:, :64]).all()
