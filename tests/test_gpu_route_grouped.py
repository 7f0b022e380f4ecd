"""Grouped softmax / sigmoid routing on the GPU against a plain 64-bit form.

Ids are compared exactly: the inputs are drawn until no token's order hangs on less than 2^-16 of a
key (equal logits with equal biases are exact ties and stay). Weights: exp 2 units of 2^-24, the
sums of at most E and K terms in trees or in order, two divisions and two products: within
(K + 40) 2^-24 of the value, doubled."""
import numpy as np
import pytest
import torch

import block_reference as ref
from gpu_helpers import dev, host

pytestmark = pytest.mark.gpu


def run(moe, x, bias, K, scoring="sigmoid", groups=1, kept=1, rule="top2", renorm=True, scale=1.0):
    ids, w, wb = moe.topk_route_grouped(
        dev(x.astype(np.float32)), None if bias is None else dev(bias.astype(np.float32)), K, n_group=groups, topk_group=kept,
        scoring=moe.SCORE_SIGMOID if scoring == "sigmoid" else moe.SCORE_SOFTMAX,
        group_rule=moe.GROUP_TOP2 if rule == "top2" else moe.GROUP_MAX, renormalize=renorm, scale=scale)
    assert torch.equal(wb, w.to(torch.bfloat16))
    return host(ids), host(w)


def check(moe, x, bias, K, **kw):
    ids, w = run(moe, x, bias, K, **kw)
    opts = dict(scoring="sigmoid", groups=1, kept=1, rule="top2", renorm=True, scale=1.0)
    opts.update(kw)
    for t in range(x.shape[0]):
        eid, ew = ref.route(x[t], bias, K, **opts)
        np.testing.assert_array_equal(ids[t], eid, err_msg=f"token {t}")
        assert np.all(np.abs(w[t] - ew) <= 2 * (K + 40) * 2.0 ** -24 * np.abs(ew) + 2.0 ** -126), f"token {t}"


def separated(rng, T, E, bias, scoring, groups, rule):
    """Logits of a BF16 router whose keys, and groups' values, differ by nothing or by enough."""
    def bad(x):
        x64 = x.astype(np.float64)
        s = 1 / (1 + np.exp(-x64)) if scoring == "sigmoid" else np.exp(x64 - x64.max()) / np.exp(x64 - x64.max()).sum()
        key = s if bias is None else s + bias.astype(np.float64)
        by = -np.sort(-key.reshape(groups, -1), axis=1)
        v = by[:, :2].sum(1) if rule == "top2" else by[:, 0]
        for k in (np.sort(key), np.sort(v)):
            d = np.diff(k)
            if np.any((d > 0) & (d < 2.0 ** -16 * np.abs(k[1:]))):
                return True
        return False

    out = []
    while len(out) < T:
        x = ref.bf16(rng.normal(0, 1, E))
        if not bad(x):
            out.append(x)
    return np.array(out)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E,K,groups,kept,rule", [
    (1, 1, 1, 1, "max"), (8, 8, 1, 1, "max"), (33, 5, 1, 1, "max"), (64, 6, 8, 3, "max"), (64, 8, 8, 4, "top2"), (60, 4, 4, 1, "max"),
    (66, 7, 6, 2, "top2"), (128, 16, 16, 16, "top2"), (16, 2, 16, 2, "top2"), (100, 25, 4, 1, "top2"), (96, 32, 3, 2, "max")])
def test_route(moe, scoring, with_bias, E, K, groups, kept, rule):
    rng = np.random.default_rng(E * 100 + K)
    bias = ref.bf16(rng.normal(0, 0.1, E)) if with_bias else None
    x = separated(rng, 9, E, bias, scoring, groups, rule)
    check(moe, x, bias, K, scoring=scoring, groups=groups, kept=kept, rule=rule, renorm=E % 2 == 0, scale=2.5 if K > 4 else 1.0)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,kept", [(256, 8, 4), (384, 1, 1), (896, 1, 1), (896, 16, 5), (1000, 8, 2), (1024, 32, 7), (2048, 64, 9), (4096, 4, 2)])
def test_route_many_experts(moe, scoring, E, groups, kept):
    """Logits spread so far apart that every key differs (a permutation of an even grid)."""
    rng = np.random.default_rng(E)
    x = np.stack([rng.permutation(np.linspace(-4, 4, E)) for _ in range(5)]).astype(np.float32).astype(np.float64)
    check(moe, x, None, 16, scoring=scoring, groups=groups, kept=kept, rule="max")


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 63, 1020])
def test_sigmoid_without_groups_is_topk_route(moe, T):
    rng = np.random.default_rng(T)
    x = dev(rng.normal(0, 1, (T, 896)).astype(np.float32))
    bias = dev(rng.normal(0, 0.01, 896).astype(np.float32))
    a = moe.topk_route_grouped(x, bias, 16, scale=2.5)
    b = moe.topk_route(x, bias, 16, scale=2.5)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_ties_go_to_the_lowest_index(moe):
    x = np.zeros((3, 64))
    x[1, 40:] = 1.0
    x[2, ::2] = 2.0
    for scoring in ("sigmoid", "softmax"):
        check(moe, x, None, 6, scoring=scoring, groups=8, kept=2, rule="top2")
        check(moe, x, None, 6, scoring=scoring, groups=8, kept=2, rule="max")
        check(moe, x, None, 32, scoring=scoring)


@pytest.mark.parametrize("E", [300, 896, 1024])
def test_more_ties_than_candidates(moe, E):
    """More experts at the bound than are ranked against each other: the lowest indices, in order."""
    x = np.zeros((3, E))
    x[1, 100:] = 1.0
    x[2, 200:205] = 3.0
    for scoring in ("sigmoid", "softmax"):
        check(moe, x, None, 16, scoring=scoring)
        check(moe, x, np.zeros(E), 16, scoring=scoring)
        check(moe, x, None, 16, scoring=scoring, groups=4, kept=2, rule="top2")


def test_masked_and_special_logits(moe):
    """Rows whose mask leaves few, one or no experts (-inf or the type's lowest value), NaN, +inf."""
    low = float(np.finfo(np.float32).min)
    rng = np.random.default_rng(0)
    x = ref.bf16(rng.permutation(np.linspace(-3, 3, 64 * 12)).reshape(12, 64) * 4)
    x[0] = -np.inf
    x[1] = low
    x[2] = np.nan
    x[3, 5:] = -np.inf
    x[4, 5:] = low
    x[5, 10:] = np.nan
    x[6, [3, 50]] = np.inf
    x[7] = -np.inf
    x[7, 61] = 1.0
    x[8, :8] = np.nan
    x[9, 1::2] = -np.inf
    x[10, 7] = np.inf
    x[10, 8:] = -np.inf
    for scoring in ("sigmoid", "softmax"):
        for groups, kept, rule in ((1, 1, "max"), (8, 2, "top2"), (8, 3, "max")):
            ids, w = run(moe, x, None, 8, scoring=scoring, groups=groups, kept=kept, rule=rule, scale=2.5)
            assert np.isfinite(w).all()
            for t in range(12):
                eid, ew = ref.route(x[t], None, 8, scoring, groups, kept, rule, True, 2.5)
                # (scores that underflow 32 bits but not 64 order by value there and by index here)
                if scoring == "sigmoid" or t not in (5, 8, 11):
                    same = ids[t] == eid
                    assert np.all(same | (ew < 1e-30)), (scoring, groups, t)
                assert np.all(np.abs(w[t] - ew) <= 1e-5 * np.abs(ew) + 1e-30), (scoring, groups, t)
    bias = np.zeros(64)
    bias[::3] = -np.inf
    bias[1] = np.nan
    ids, w = run(moe, x[11:12], bias, 8, scoring="sigmoid")
    eid, _ = ref.route(x[11], bias, 8, "sigmoid", 1, 1, "max", True, 1.0)
    np.testing.assert_array_equal(ids[0], eid)


def test_optional_outputs_and_stream(moe):
    rng = np.random.default_rng(1)
    x = dev(rng.normal(0, 1, (7, 96)).astype(np.float32))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ids, w, wb = moe.topk_route_grouped(x, None, 5, n_group=4, topk_group=2, want_bf16=False, stream=s)
    s.synchronize()
    assert wb is None
    ids2, w2, _ = moe.topk_route_grouped(x, None, 5, n_group=4, topk_group=2)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)


def test_refusals(moe):
    x = torch.zeros(2, 60, device="cuda")
    for kw in (dict(K=0), dict(K=4, n_group=7), dict(K=4, n_group=4, topk_group=5), dict(K=16, n_group=4, topk_group=1),
               dict(K=4, scoring=2), dict(K=4, group_rule=2), dict(K=4, n_group=0), dict(K=33)):
        with pytest.raises(moe.MoeError):
            moe.topk_route_grouped(x, None, **kw)
    with pytest.raises(ValueError):
        moe.topk_route_grouped(x, torch.zeros(59, device="cuda"), 4)
    with pytest.raises(TypeError):
        moe.topk_route_grouped(x.half(), None, 4)
    assert moe.topk_route_grouped(torch.zeros(0, 60, device="cuda"), None, 4)[0].shape == (0, 4)
