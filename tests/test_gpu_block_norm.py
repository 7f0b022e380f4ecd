"""The block norm on the GPU against a plain 64-bit form.

Tolerances. A mean of squares in FP32 (a thread's columns in order, then trees) is off by at most
64 units of 2^-24 for the widths here, its root by half of that; with the products u is within
2^-18 of its value, h within 2^-18 (|residual| + |alpha gate u|), and n within 2^-17 of
|next_weight| times that, over the row's root. A BF16 output adds half a step, 2^-8 of its value;
a code is within half a step of E4M3 of n, plus that error."""
import numpy as np
import pytest
import torch

import block_reference as ref
from gpu_helpers import host

pytestmark = pytest.mark.gpu


def case(seed, T, H, f32, gate, post):
    rng = np.random.default_rng(seed)
    y = ref.bf16(rng.normal(0, 3, (T, H)))
    r = rng.normal(0, 2, (T, H))
    r = r.astype(np.float32).astype(np.float64) if f32 else ref.bf16(r)
    shape = {"none": None, "token": (T, 1), "channel": (H,), "full": (T, H)}[gate]
    g = None if shape is None else ref.bf16(rng.normal(1, 0.5, shape))
    return y, r, ref.bf16(1 + 0.1 * rng.normal(0, 1, H)) if post else None, g, ref.bf16(1 + 0.1 * rng.normal(0, 1, H))


def run(moe, y, r, post, g, nxt, alpha, eps, f32, quantize, **kw):
    t = ref.to_bf16_cuda
    residual = torch.from_numpy(r.astype(np.float32)).cuda() if f32 else t(r)
    return moe.block_norm(t(y), residual, t(nxt), post_weight=None if post is None else t(post),
                          gate=None if g is None else t(g), alpha=alpha, eps=eps, quantize=quantize, **kw)


def check(moe, y, r, post, g, nxt, alpha, eps, f32, quantize):
    h, n, q, s = run(moe, y, r, post, g, nxt, alpha, eps, f32, quantize)
    eh, en = ref.block_norm(y, r, post, g, nxt, alpha, eps)
    mag = np.abs(r) + np.abs(eh - r)
    th = 2.0 ** -18 * mag
    assert np.all(np.abs(h.double().cpu().numpy() - eh) <= th + (0 if f32 else 2.0 ** -8 * np.abs(eh)) + 1e-37)
    inv = 1 / np.sqrt((eh * eh).mean(1, keepdims=True) + eps)
    tn = 2.0 ** -17 * np.abs(nxt) * mag * inv + 1e-37
    assert np.all(np.abs(n.double().cpu().numpy() - en) <= tn + 2.0 ** -8 * np.abs(en))
    if quantize:
        s64 = host(s).astype(np.float64)
        amax = ref.block_amax(en)
        ta = ref.block_amax(tn)
        live = amax > 0
        assert np.all(np.abs(s64 - amax / 448)[live] <= (ta / 448 + 2.0 ** -23 * amax / 448)[live])
        assert np.all(s64[~live] == 1)
        got, step = ref.DECODE[host(q)] * ref.expand(s64, en.shape[1]), ref.expand(s64, en.shape[1])
        assert np.all(np.abs(got - en) <= np.maximum(np.abs(en) / 16, step * 2.0 ** -10) * (1 + 2.0 ** -9) + tn)
    else:
        assert q is None and s is None


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 136), (2, 1000), (5, 3584)])
def test_block_norm(moe, T, H, gate, post, f32):
    check(moe, *case(T + H, T, H, f32, gate, post), alpha=0.7, eps=1e-6, f32=f32, quantize=True)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,H", [(1, 7168), (2, 4096), (3, 4104), (2, 8192), (2, 8200), (1, 16384), (700, 256), (40, 32)])
def test_widths(moe, T, H, f32):
    check(moe, *case(T + H, T, H, f32, "full", True), alpha=-1.25, eps=1e-5, f32=f32, quantize=T % 2 == 1)


@pytest.mark.parametrize("f32", [False, True])
def test_zero_rows(moe, f32):
    """A row of zeros: eps keeps the roots finite, n is 0 with scale 1; with eps 0 its n is NaN (0 times infinity)."""
    y, r, post, g, nxt = case(3, 3, 264, f32, "full", True)
    y[1], r[1] = 0.0, 0.0
    check(moe, y, r, post, g, nxt, alpha=0.5, eps=1e-6, f32=f32, quantize=True)
    h, n, q, s = run(moe, y, r, post, g, nxt, 0.5, 0.0, f32, True)
    assert torch.isnan(n[1]).all() and torch.isfinite(n[0]).all() and torch.isfinite(n[2]).all()
    assert torch.isnan(s[1]).all() and (q[1] == 0x7F).all()


def test_in_place_and_row_stride(moe):
    """h over the residual; y a slice of wider rows."""
    y, r, post, g, nxt = case(5, 50, 520, True, "channel", True)
    t = ref.to_bf16_cuda
    expect = run(moe, y, r, post, g, nxt, 0.7, 1e-6, True, True)
    wide = np.full((50, 1048), 1e30)
    wide[:, 264:784] = y
    residual = torch.from_numpy(r.astype(np.float32)).cuda()
    got = moe.block_norm(t(wide)[:, 264:784], residual, t(nxt), post_weight=t(post), gate=t(g), alpha=0.7, eps=1e-6, h=residual, quantize=True)
    assert got[0] is residual
    for u, v in zip(expect, got):
        assert torch.equal(u, v)


def test_other_stream(moe):
    y, r, post, g, nxt = case(6, 9, 640, False, "token", True)
    t = [ref.to_bf16_cuda(v) for v in (y, r, nxt, post, g)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = moe.block_norm(t[0], t[1], t[2], post_weight=t[3], gate=t[4], stream=s)
    s.synchronize()
    expect = moe.block_norm(t[0], t[1], t[2], post_weight=t[3], gate=t[4])
    assert torch.equal(got[0], expect[0]) and torch.equal(got[1], expect[1])


def test_refusals(moe):
    bf = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError):
        moe.block_norm(bf(2, 12), bf(2, 12), bf(12))
    with pytest.raises(moe.MoeError):
        moe.block_norm(bf(2, 16392), bf(2, 16392), bf(16392))
    with pytest.raises(moe.MoeError):
        moe.block_norm(bf(2, 16), bf(2, 16), bf(16), eps=-1.0)
    with pytest.raises(moe.MoeError):
        moe.block_norm(bf(2, 20)[:, :16], bf(2, 16), bf(16))
    with pytest.raises(ValueError):
        moe.block_norm(bf(2, 16), bf(2, 16), bf(16), gate=bf(2))
    with pytest.raises(ValueError):
        moe.block_norm(bf(2, 24), bf(2, 16), bf(16))
    with pytest.raises(TypeError):
        moe.block_norm(bf(2, 16), bf(2, 16).half(), bf(16))
    with pytest.raises(ValueError):
        moe.block_norm(bf(2, 16), bf(2, 16), bf(8))
    assert moe.block_norm(bf(0, 16), bf(0, 16), bf(16))[1].shape == (0, 16)
