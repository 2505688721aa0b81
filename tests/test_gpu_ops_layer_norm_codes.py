"""The layer norm's choices of code, and what a wrong one is told."""
import pytest
import torch

from sharded_optimizer_step_zero_amd import ops

pytestmark = pytest.mark.gpu


def test_a_wrong_code_is_told_every_right_one():
    x, w = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    for code in ("fp4", "E2M1", 4, ["e2m1"]):
        with pytest.raises(ValueError, match="code: .*'e4m3', 'e5m2', 'e2m1'"):
            ops.layer_norm(x, w, code=code)
    with pytest.raises(ValueError, match="code: .*'e4m3', 'e5m2'\\)"):
        ops.norm(x, w, code="e2m1")


@pytest.mark.parametrize("code, dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2),
                                         ("e2m1", torch.float4_e2m1fn_x2), (None, None)])
def test_codes_have_their_type(code, dtype):
    r = ops.layer_norm(torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda"), code=code)
    assert (r.codes.dtype if code else r.codes) == dtype
