"""Calls that the documentation allows or refuses, beside those of test_step_gpu.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, F64, I8, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int8, torch.int32


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import conv_bn_silu_amd
    return conv_bn_silu_amd


def test_a_wrong_sum_is_called_by_its_name(ops):
    x, r = torch.zeros(4, 64, dtype=BF16, device="cuda"), torch.zeros(4, 64, dtype=BF16, device="cuda")
    with pytest.raises(TypeError, match="^sum_out"):
        ops.add_rms_norm(x, None, r, sum_out=torch.zeros(4, 64, device="cuda"))
    for bad in (r[:3], torch.zeros(4, 128, dtype=BF16, device="cuda")[:, ::2], r.cpu()):
        with pytest.raises(ValueError, match="^sum_out"):
            ops.add_rms_norm(x, None, r, sum_out=bad)
    with pytest.raises(ValueError, match="^out"):
        ops.add_rms_norm(x, None, r, out=r[:3])
