"""Sums of the BF16 products over a long K (of a weight's gradient: over many rows)."""
import pytest
import torch

import linear_reference as ref
from test_gpu_linear import BF, F32, check_gated, check_gated_backward, check_linear, check_linear_backward, rand

pytestmark = pytest.mark.gpu

LONG = 1 << 20


def positive(g, rows, cols):
    """Values of one sign, each row at a scale of its own, so that sums grow all the way and results lie anywhere
    between two powers of two."""
    return ((0.5 + 0.5 * torch.rand(rows, cols, generator=g, device="cuda")) * torch.exp2(torch.rand(rows, 1, generator=g, device="cuda"))).to(BF)


def centred(got, expect):
    """Rounding to BF16 is off by at most 2^-8 of a value, evenly to both sides: 2^-8 / sqrt(12) rms, of n values' mean
    5 sigma / sqrt(n). What the tensor core cuts off a running sum goes one way, some 2e-8 of it for every 16 values of K: of a sum of
    8192 that is 1e-5, of 2^20 6e-4 or more."""
    off = ((got.double() - expect) / expect).mean().abs()
    assert off <= 5 * 2.0 ** -8 / 12 ** 0.5 / got.numel() ** 0.5 + 1e-5, float(off)


def test_gradient_of_weights_over_many_rows(moe):
    g = torch.Generator(device="cuda").manual_seed(0)
    dout, x, w = positive(g, 64, LONG).t().contiguous(), positive(g, 64, LONG).t().contiguous(), rand(g, 64, 64)
    dw = moe.bf16_linear_backward(dout, x, w, want_dx=False)[1]
    centred(dw, dout.double().t() @ x.double())
    pre = torch.ones_like(dout)
    centred(moe.bf16_linear_backward(dout, x, w, pre, moe.ACT_RELU)[1], dout.double().t() @ x.double())


@pytest.mark.parametrize("t", [16, 300])
def test_rows_of_many_columns(moe, t):
    g = torch.Generator(device="cuda").manual_seed(t)
    x, w = positive(g, t, LONG), positive(g, 256, LONG)
    exact = x.double() @ w.double().t()
    centred(moe.bf16_linear(x, w)[0], exact)
    bias, residual = rand(g, 256, scale=1e4), rand(g, t, 256, scale=1e4)
    out, pre = moe.bf16_linear(x, w, bias=bias, residual=residual, activation=moe.ACT_RELU, want_pre=True)
    centred(pre, exact + bias.double())
    centred(out, exact + bias.double() + residual.double())
    out, pre = moe.bf16_gated_linear(x, w, activation=moe.ACT_NONE, want_pre=True)
    centred(pre, exact)
    expect = exact[:, :128] * exact[:, 128:]
    off = ((out.double() - expect) / expect).mean().abs()
    assert off <= 5 * 2.0 ** -8 / 12 ** 0.5 / out.numel() ** 0.5 + 2e-5, float(off)


@pytest.mark.parametrize("t,n", [(70, 130), (300, 515), (1500, 2050), (2000, 1536)])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_epilogues_behind_long_sums(moe, t, n, pad):
    k = 8264  # (a block and a bit beyond what a sum takes whole)
    check_linear(moe, t, n, k, "gelu", BF, F32, BF, True, pad)
    check_linear(moe, t, n, k, "none", F32, BF, BF, False, pad)
    check_gated(moe, t, n // 2, k, "silu", True, pad)


@pytest.mark.parametrize("t,n,k", [(9001, 130, 72), (8200, 600, 521)])
def test_gradients_over_long_batches(moe, t, n, k):
    for dtypes in ((BF, BF), (F32, BF), (BF, F32)):
        check_linear_backward(moe, t, n, k, "none", dtypes)
    check_linear_backward(moe, t, n, k, "silu", odd_dout=True, pad=1)
    check_gated_backward(moe, t, n // 2, k)


@pytest.mark.parametrize("t,n", [(1, 520), (40, 1000), (600, 520), (600, 515)])
@pytest.mark.parametrize("scale", [1.0, 100.0])
def test_fp32_sums_with_bias_and_residual(moe, t, n, scale):
    """As plain products' (1e-6 of the whole, rms), and the additions of the 14 runs, the bias and the residual
    to the sum: 16 roundings of at most 2^-24 of it, evenly to both sides, below 4 * 2^-24 rms."""
    g = torch.Generator(device="cuda").manual_seed(n)
    k = 7168
    x, w = rand(g, t, k), rand(g, n, k, scale=k ** -0.5)
    z = x.double() @ w.double().t()
    for bias, residual in ((F32, None), (BF, None), (None, F32), (None, BF), (F32, F32), (BF, BF)):
        b = None if bias is None else rand(g, n, dtype=bias, scale=scale)
        r = None if residual is None else rand(g, t, n, dtype=residual, scale=scale)
        for name in ("none", "relu"):
            out, _ = moe.bf16_linear(x, w, bias=b, residual=r, activation=moe.ACT_RELU if name == "relu" else moe.ACT_NONE, out_dtype=F32)
            expect = ref.linear(x.double(), w.double(), None if b is None else b.double(), name, None if r is None else r.double())[0]
            added = (0 if b is None else b.double().norm() * t ** 0.5) + (0 if r is None else r.double().norm())
            assert (out.double() - expect).norm() <= 1e-6 * z.norm() + 2.0 ** -22 * added
