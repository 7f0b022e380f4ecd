"""The example block: every stage against its 64-bit form on that stage's own inputs, eagerly and
replayed from a CUDA graph over other inputs.

Tolerances: those of the operators' own tests; the two products' BF16 outputs are within
(K + 8) 2^-23 of the terms' magnitudes and 2^-8 of the value, codes within half a step."""
import os
import sys

import numpy as np
import pytest
import torch

import block_reference as ref
from gpu_helpers import host

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def codes_hold(q, s, v):
    s64 = host(s).astype(np.float64)
    got, step = ref.DECODE[host(q)] * ref.expand(s64, v.shape[1]), ref.expand(s64, v.shape[1])
    assert np.all(np.abs(got - v) <= np.maximum(np.abs(v) / 16, step * 2.0 ** -10) * (1 + 2.0 ** -9))


def product_holds(out, a, sa, w, sw):
    ra, rw = ref.real_rows(host(a), host(sa)), ref.real_weights(host(w), host(sw))
    exact, mags = ra @ rw.T, np.abs(ra) @ np.abs(rw).T
    assert np.all(np.abs(f64(out) - exact) <= (ra.shape[1] + 8) * 2.0 ** -23 * mags + 2.0 ** -8 * np.abs(exact))


def stages_hold(b, y, residual):
    h, n = ref.block_norm(f64(y), f64(residual), f64(b.post_norm), None, f64(b.next_norm), b.alpha, b.eps)
    mag = np.abs(f64(residual)) + np.abs(h - f64(residual))
    assert np.all(np.abs(f64(b.h) - h) <= 2.0 ** -18 * mag)
    inv = 1 / np.sqrt((h * h).mean(1, keepdims=True) + b.eps)
    tn = 2.0 ** -17 * np.abs(f64(b.next_norm)) * mag * inv
    assert np.all(np.abs(f64(b.n) - n) <= tn + 2.0 ** -8 * np.abs(n))
    # router logits of BF16 rows, FP32 sums
    x, g = f64(b.n), f64(b.gate)
    assert np.all(np.abs(f64(b.logits) - x @ g.T) <= 1e-5 * (np.abs(x) @ np.abs(g).T))
    # the choice, from those logits: keys at least as large as any expert's left out (to 2^-20)
    s = 1 / (1 + np.exp(-f64(b.logits)))
    key, ids = s + f64(b.bias), host(b.ids)
    size = b.E // b.n_group
    for t in range(b.T):
        assert len(set(ids[t])) == b.K
        groups = np.sort(key[t].reshape(b.n_group, size), axis=1)[:, -2:].sum(1)
        kept = set(ids[t] // size)
        assert len(kept) <= b.topk_group
        assert all(groups[k] >= np.sort(groups)[-b.topk_group] - 2.0 ** -20 for k in kept)
        w = s[t][ids[t]]
        assert np.all(np.diff(key[t][ids[t]]) <= 2.0 ** -20)
        assert np.all(np.abs(host(b.weights)[t] - b.scale * w / w.sum()) <= 1e-5)
    offsets, pairs = host(b.offsets), host(b.pairs)
    assert offsets[-1] == b.T * b.K
    product_holds(b.latent, b.q, b.s, b.w_down, b.s_down)
    codes_hold(b.lq, b.ls, f64(b.latent))
    for e in range(b.E):
        pos = np.arange(offsets[e], offsets[e + 1])
        assert np.all(ids.reshape(-1)[pairs[pos]] == e)
        if pos.size:
            at, p = torch.from_numpy(pos).cuda(), torch.from_numpy(pairs[pos].astype(np.int64)).cuda()
            product_holds(b.gu[at], b.lq[p // b.K], b.ls[p // b.K], b.w_gu[e], b.s_gu[e])
            product_holds(b.rows[p], b.aq[at], b.as_[at], b.w_dn[e], b.s_dn[e])
    codes_hold(b.aq, b.as_, ref.silu_up(f64(b.gu)))
    rows, w = f64(b.rows).reshape(b.T, b.K, b.L), f64(b.weights_bf16)[..., None]
    routed = (rows * w).sum(1)
    assert np.all(np.abs(f64(b.routed) - routed) <= 2.0 ** -8 * np.abs(routed) + 2.0 ** -18 * np.abs(rows * w).sum(1))
    codes_hold(b.rq, b.rs, f64(b.routed))
    product_holds(b.y, b.rq, b.rs, b.w_up, b.s_up)


def inputs(seed, T, H):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (3 * torch.randn(T, H, generator=g, device="cuda")).to(torch.bfloat16), 2 * torch.randn(T, H, generator=g, device="cuda")


@pytest.mark.parametrize("T,H,L,F,E,K,G,KG", [(1, 512, 256, 128, 16, 4, 4, 2), (9, 640, 272, 144, 24, 3, 6, 2), (70, 512, 384, 128, 8, 4, 1, 1),
                                              (300, 256, 256, 256, 8, 4, 2, 1)])
def test_stages(moe, T, H, L, F, E, K, G, KG):
    from moe_block import MoeBlock

    b = MoeBlock(T, H, L, F, E, K, n_group=G, topk_group=KG, alpha=0.7)
    y, residual = inputs(T, T, H)
    b.run(y, residual)
    stages_hold(b, y, residual)
    assert moe.device_error() == 0


def test_graph(moe):
    from moe_block import MoeBlock

    b = MoeBlock(12, 512, 256, 128, 16, 4, n_group=4, topk_group=2)
    y, residual = inputs(1, 12, 512)
    b.run(y, residual)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(y, residual)
    y2, r2 = inputs(2, 12, 512)
    y.copy_(y2)
    residual.copy_(r2)
    g.replay()
    torch.cuda.synchronize()
    stages_hold(b, y, residual)


def test_example_runs(moe, monkeypatch, capsys):
    import moe_block

    monkeypatch.setattr(sys, "argv", ["moe_block.py", "8"])
    moe_block.main()
    assert "us a block" in capsys.readouterr().out
