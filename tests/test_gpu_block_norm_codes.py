"""The block norm's codes where its values leave the usual range: blocks of very small values, rows
whose sum of squares overflows, infinities. The codes are those of n before its rounding to BF16, by
the rule of fp8_block_quantize_rows; few rows (one CTA each) and streamed ones.

Tolerances: the post norm is of zeros here, so h is the residual itself. A mean of squares is within
2^-18 of its value for these widths, its root within 2^-19 (rsqrtf's 2 units included); n adds two
roundings, the scale one, so a code lies within half a step (2^-4 of a normal code's value, 2^-10 of
the scale's unit below) of n, widened by 2^-9 as a tie may fall to either side."""
import numpy as np
import pytest
import torch

import block_reference as ref
from gpu_helpers import host

pytestmark = pytest.mark.gpu

H = 520  # four blocks and one of 8 columns
TINY = 2.0 ** -110


def run(moe, r, nxt, eps, f32, rows):
    t = ref.to_bf16_cuda
    reps = -(-rows // r.shape[0])
    full = np.tile(r, (reps, 1))[:rows]
    residual = torch.from_numpy(full.astype(np.float32)).cuda()
    if not f32:
        residual = residual.to(torch.bfloat16)
    y = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
    h, n, q, s = moe.block_norm(y, residual, t(nxt), post_weight=t(np.ones(H)), eps=eps, quantize=True)
    assert np.array_equal(h.double().cpu().numpy(), residual.double().cpu().numpy(), equal_nan=True)
    n, q, s = n.double().cpu().numpy(), host(q), host(s).astype(np.float64)
    k = r.shape[0]
    for at in range(k, rows):  # a row's result does not hang on where it lies
        assert np.array_equal(q[at], q[at % k]) and np.array_equal(s[at], s[at % k], equal_nan=True) and np.array_equal(n[at], n[at % k], equal_nan=True)
    return residual.double().cpu().numpy()[:k], n[:k], q[:k], s[:k]


@pytest.mark.parametrize("rows", [4, 900])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("eps", [1e-6, 1e-9, 1e-12])
def test_small_blocks(moe, eps, f32, rows):
    rng = np.random.default_rng(int(-np.log10(eps)))
    r = rng.normal(0, 1, (4, H)) * np.array([7e-7, 1e-4, 3e-5, 1e-9])[:, None]
    for i, top in enumerate((1e-37, 1.2e-36, 3e-38, 4e-39)):
        r[i, 128:256] = 0.0
        r[i, 130:136] = top * np.array([1.0, 0.5, -0.5, 0.25, -1.0, 0.125])
    r[2, 512:] = 0.0
    r[2, 515] = 2e-38
    r[3, 384:512] = 0.0
    nxt = ref.bf16(1 + 0.1 * rng.normal(0, 1, H))
    h, n, q, s = run(moe, r, nxt, eps, f32, rows)
    en = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * nxt
    assert np.all(np.abs(n - en) <= (2.0 ** -8 + 2.0 ** -17) * np.abs(en) + 2.0 ** -133)
    amax = ref.block_amax(en)
    es = np.where(amax == 0, 1.0, np.maximum(amax, TINY) / 448)
    assert np.all(np.abs(s - es) <= 2.0 ** -17 * es)
    got, step = ref.DECODE[q] * ref.expand(s, H), ref.expand(s, H)
    assert np.all(np.abs(got - en) <= np.maximum(np.abs(en) / 16, step * 2.0 ** -10) * (1 + 2.0 ** -9))
    assert np.all(q[h == 0] & 0x7F == 0)


@pytest.mark.parametrize("rows", [3, 900])
@pytest.mark.parametrize("f32", [False, True])
def test_rows_without_a_finite_root(moe, f32, rows):
    """A sum of squares that is infinite (one infinite value; values about 1e20) has the root 0: n is 0 wherever
    h is finite, and its codes are zeros with the scale 1; the block of the infinity is NaN."""
    rng = np.random.default_rng(9)
    r = rng.normal(0, 1, (3, H))
    r[0, 200] = np.inf
    r[1] *= 1e20
    r[2, 5], r[2, 519] = -np.inf, np.nan
    h, n, q, s = run(moe, r, ref.bf16(1 + 0.1 * rng.normal(0, 1, H)), 1e-6, f32, rows)
    bad = np.zeros((3, 5), bool)
    bad[0, 1] = True
    bad[2] = True  # (the sum is NaN, and with it the root)
    cols = np.repeat(bad, 128, axis=1)[:, :H]
    assert np.isnan(s[bad]).all() and (q[cols] == 0x7F).all()
    assert (s[~bad] == 1).all() and (q[~cols] & 0x7F == 0).all()
    assert (n[~cols] == 0).all()
