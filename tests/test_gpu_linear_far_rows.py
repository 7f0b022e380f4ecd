"""Gradients over nothing are zeros in rows however far apart, and nowhere else."""
import pytest
import torch

from test_gpu_linear import BF, F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,step", [(F32, (1 << 29) + 64), (BF, (1 << 30) + 64), (F32, 1 << 20)])
def test_zeros_in_far_rows(moe, dtype, step):
    """(rows 2^31 bytes and more apart, and fewer)"""
    e = lambda *s: torch.ones(*s, dtype=BF, device="cuda")
    whole = torch.full((2 * step + 64,), 77.0, dtype=dtype, device="cuda")
    far, beside = torch.as_strided(whole, (3, 24), (step, 1)), torch.as_strided(whole, (3, 40), (step, 1), 24)
    moe.bf16_linear_backward(e(3, 0), e(3, 24), e(0, 24), dx=far, want_dw=False)
    assert not far.any() and (beside == 77).all()
    far.fill_(77)
    moe.bf16_linear_backward(e(0, 3), e(0, 24), e(3, 24), dw=far, want_dx=False)
    assert not far.any() and (beside == 77).all()
    far = torch.as_strided(whole, (2, 24), (step, 1))
    far.fill_(77)
    moe.bf16_gated_linear_backward(e(0, 1), e(0, 24), e(2, 24), e(0, 2), dw=far, want_dx=False)
    assert not far.any() and (beside == 77).all()
    assert moe.device_error() == 0
