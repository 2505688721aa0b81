"""zs_layer_norm_forward with the sum written over x or over the residual, which it allows."""
import pytest
import torch

from sharded_optimizer_step_zero_amd import ops

pytestmark = pytest.mark.gpu
DT = {torch.float32: ops.ZS_F32, torch.bfloat16: ops.ZS_BF16, torch.float16: ops.ZS_F16}


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("code", [None, "e4m3", "e2m1"])
@pytest.mark.parametrize("rows, width, stride", [(1, 1, 1), (70, 5, 9), (33, 515, 517), (300, 1001, 1001), (41, 8192, 8200),
                                                 (9, 8203, 8203), (3, 40001, 40008)])
def test_the_sum_over_an_input(dtype, code, rows, width, stride):
    g = torch.Generator(device="cuda").manual_seed(rows + width)
    big = torch.randn(2, rows, stride, generator=g, device="cuda").to(dtype)
    x, residual = big[0, :, :width], big[1, :, :width]
    w, b = (torch.randn(width, generator=g, device="cuda").to(dtype) for _ in range(2))
    want = ops.layer_norm(x, w, b, residual=residual, code=code, group=32 if code else None)
    keep = big.clone()
    for over in (0, 1):
        big.copy_(keep)
        y = torch.empty(rows, width, dtype=dtype, device="cuda")
        mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
        codes = scales = None
        if code:
            codes = torch.zeros_like(want.codes.view(torch.uint8))
            scales = torch.zeros_like(want.scales.view(torch.uint8))
        ops.zs_layer_norm_forward(x.data_ptr(), stride, residual.data_ptr(), stride, w.data_ptr(), b.data_ptr(),
                                  big[over].data_ptr(), stride, y.data_ptr(), width, codes.data_ptr() if code else None,
                                  scales.data_ptr() if code else None, mean.data_ptr(), rstd.data_ptr(), rows, width, 1e-5,
                                  DT[dtype], {None: 0, "e4m3": ops.ZS_E4M3, "e2m1": ops.ZS_E2M1}[code], 32,
                                  torch.cuda.current_stream().cuda_stream)
        assert torch.equal(big[over, :, :width], want.sum) and torch.equal(y, want.y)
        assert torch.equal(mean, want.mean) and torch.equal(rstd, want.rstd)
        if code:
            assert torch.equal(codes, want.codes.view(torch.uint8)) and torch.equal(scales, want.scales.view(torch.uint8))
        # the other input and what lies between the rows stay as they are
        assert torch.equal(big[1 - over], keep[1 - over]) and torch.equal(big[over, :, width:], keep[over, :, width:])
