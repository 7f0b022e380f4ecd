"""silu as fp8_block_quantize_swiglu computes it, over every finite BF16 gate: the only value of its block, with
up = 1, it is 448 times the block's scale.

Tolerance, in units of the value: the exponent's argument y = -gate log2 e is rounded once, half a unit of its
last place, and its constant is off by 2^-26 of itself, both times ln 2; ex2.approx 2^-22 (documented: 2 units),
both times e / (1 + e); the sum 2^-24, rcp.approx 2^-23 (documented: 1 unit), the product and the scale's
division 2^-24 each. That is 1.45 x 2^-20 at most to |gate| = 12."""
import numpy as np
import pytest
import torch

from gpu_helpers import host

pytestmark = pytest.mark.gpu


def test_silu_over_all_gates(moe):
    g = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    g = g[torch.isfinite(g)]
    x = torch.zeros(g.numel(), 16, dtype=torch.bfloat16)
    x[:, 0], x[:, 8] = g, 1.0
    q, s = moe.fp8_block_quantize_swiglu(x.cuda())
    g = g.double().numpy()
    with np.errstate(over="ignore"):
        silu = np.abs(g / (1 + np.exp(-g)))
    got = host(s)[:, 0].astype(np.float64) * 448
    live = silu >= 2.0 ** -109  # (below 2^-110 the scale is that of 2^-110)
    y = np.abs(g) * np.log2(np.e)
    half_unit = np.exp2(np.floor(np.log2(np.maximum(y, 2.0 ** -126))) - 24)
    with np.errstate(over="ignore"):
        share = 1 / (1 + np.exp(g))  # e / (1 + e), what an error of e counts for
    tol = share * (np.log(2) * (half_unit + 2.0 ** -26 * y) + 2.0 ** -22) + 2.0 ** -24 + 2.0 ** -23 + 2.0 ** -24 + 2.0 ** -24
    err = np.abs(got - silu) / np.maximum(silu, 2.0 ** -109)
    for most in (12, 64):
        m = live & (np.abs(g) <= most)
        print(f"largest error to |gate| = {most}: {err[m].max() * 2 ** 20:.2f} x 2^-20, at {g[m][err[m].argmax()]}")
    assert np.all(err[live] <= tol[live])
    assert np.all(tol[np.abs(g) <= 12] <= 1.45 * 2.0 ** -20)
    small = silu < 2.0 ** -111
    assert np.all((host(s)[small, 0] == np.float32(2.0 ** -110 / 448)) | (host(s)[small, 0] == 1))
    assert (host(q)[:, 1:] & 0x7F == 0).all()
