"""The gradients at infinities, NaN and the ends of the range: act' has its limits there."""
import math

import pytest
import torch

from test_gpu_linear import BF, F32, code

pytestmark = pytest.mark.gpu

INF = math.inf


@pytest.mark.parametrize("name", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("t", [1, 3, 70])
@pytest.mark.parametrize("pad", [0, 1])
def test_slopes_at_infinity(moe, name, t, pad):
    """1 far above, 0 far below, infinities among them: dbias and dw of dout = 1 count the rows."""
    far = torch.tensor([INF, -INF, 3e38, -3e38, 1e20, -1e20, 1e5, -1e5] * 3, device="cuda").to(BF)
    n = len(far)
    pre, dout = (torch.empty(t, n + pad, dtype=BF, device="cuda")[:, :n] for _ in range(2))
    pre[:], dout[:] = far, 1.0
    expect = (far > 0).float() * t
    x, w = torch.ones(t, 8, dtype=BF, device="cuda"), torch.ones(n, 8, dtype=BF, device="cuda")
    dx, dw, db = moe.bf16_linear_backward(dout, x, w, pre, code(moe, name), want_dbias=True, dw_dtype=F32)
    assert torch.equal(db, expect) and torch.equal(dw, expect[:, None].expand(n, 8)) and torch.equal(dx, torch.full_like(dx, n / 2))
    # the gate's half of the gated pair's: dg = dout u act'(g); du = dout act(g) has infinities of its own
    u = torch.full((t, n), 2.0, dtype=BF, device="cuda")
    both = torch.empty(t, 2 * n + pad, dtype=BF, device="cuda")[:, :2 * n]
    both[:, :n], both[:, n:] = pre, u
    dw = moe.bf16_gated_linear_backward(dout, x, torch.ones(2 * n, 8, dtype=BF, device="cuda"), both, code(moe, name), want_dx=False, dw_dtype=F32)[1]
    assert torch.equal(dw[:n], 2 * expect[:, None].expand(n, 8))
    assert moe.device_error() == 0


@pytest.mark.parametrize("t", [1, 70])
@pytest.mark.parametrize("pad", [0, 1])
def test_slopes_at_nan(moe, t, pad):
    """relu's slope is 1 where z > 0 and else 0, a NaN's too; that of the others is a NaN."""
    g = torch.Generator(device="cuda").manual_seed(t)
    n = 24
    pre, dout = (torch.empty(t, n + pad, dtype=BF, device="cuda")[:, :n] for _ in range(2))
    pre[:], dout[:] = torch.randn(t, n, generator=g, device="cuda"), torch.randn(t, n, generator=g, device="cuda")
    pre[t // 2, 5] = math.nan
    low = pre.clone()
    low[t // 2, 5] = -1.0
    x, w = (torch.randn(r, 16, generator=g, device="cuda").to(BF) for r in (t, n))
    got = moe.bf16_linear_backward(dout, x, w, pre, moe.ACT_RELU, want_dbias=True)
    for a, b in zip(got, moe.bf16_linear_backward(dout, x, w, low, moe.ACT_RELU, want_dbias=True)):
        assert torch.equal(a, b)
    gates, lows = (torch.cat([v, torch.ones_like(v)], 1) for v in (pre, low))
    w2 = torch.cat([w, w])
    a, b = (moe.bf16_gated_linear_backward(dout, x, w2, v, moe.ACT_RELU, want_dx=False)[1] for v in (gates, lows))
    assert torch.equal(a[:n], b[:n])
    for name in ("silu", "gelu", "gelu_tanh"):
        db = moe.bf16_linear_backward(dout, x, w, pre, code(moe, name), want_dbias=True)[2]
        assert db.isnan().nonzero().flatten().tolist() == [5]
