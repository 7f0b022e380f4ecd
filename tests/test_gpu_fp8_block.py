"""Block-128 E4M3 codes, their dense and per-expert products, on the GPU against plain 64-bit
forms.

Tolerances. A product's FP32 sum of n terms in any order, each step rounded or truncated to 24
bits, is off by at most (n + 8) 2^-23 times the sum of the terms' magnitudes (8: the two scales'
product, the scaling and its sum); BF16 adds half a step, 2^-8 of the value. Codes of rows follow
from FP32 operations that round correctly, so they are equal. silu(g) * up in FP32 is off by at
most 2^-20 of its value (exp 2 units, the sum, the division and the product one each, of 2^-24,
doubled), which moves a code by at most one step, and only beside a tie."""
import numpy as np
import pytest
import torch

import block_reference as ref
from gpu_helpers import dev, host

pytestmark = pytest.mark.gpu


# --- codes ------------------------------------------------------------------------

@pytest.mark.parametrize("power", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 128), (1, 7168), (3, 136), (7, 120), (33, 1000), (257, 3584), (1020, 256)])
def test_quantize_rows(moe, rows, cols, power):
    rng = np.random.default_rng(rows * 10007 + cols)
    x = ref.bf16(rng.normal(0, 1, (rows, cols)) * np.exp2(rng.integers(-30, 30, (rows, 1))))
    q, s = moe.fp8_block_quantize_rows(ref.to_bf16_cuda(x), scale_rule=moe.FP8_SCALE_POW2 if power else moe.FP8_SCALE_AMAX)
    eq, es = ref.codes32(x, power)
    np.testing.assert_array_equal(host(s), es)
    np.testing.assert_array_equal(host(q), eq)


@pytest.mark.parametrize("power", [False, True])
def test_quantize_edges(moe, power):
    """Blocks of zeros, of the smallest and largest BF16 numbers, at 448 times a power of two, and with NaN
    or infinity in one place."""
    x = np.ones((9, 256))
    x[0] = 0.0
    x[1, :128] = -0.0
    x[2] *= 2.0 ** -133            # the smallest BF16 subnormal
    x[3] *= float(torch.finfo(torch.bfloat16).max)
    x[4, 5] = 448.0
    x[5, 5] = -450.0               # one BF16 step above 448
    x[6, 7] = np.nan
    x[7, 200] = np.inf
    x[8, 200] = -np.inf
    with np.errstate(over="ignore"):
        t = ref.to_bf16_cuda(x)
    q, s = moe.fp8_block_quantize_rows(t, scale_rule=moe.FP8_SCALE_POW2 if power else moe.FP8_SCALE_AMAX)
    q, s = host(q), host(s)
    special = ~np.isfinite(x)
    bad = np.stack([special[:, :128].any(1), special[:, 128:].any(1)], 1)
    assert np.isnan(s[bad]).all() and np.isfinite(s[~bad]).all()
    assert (q[np.repeat(bad, 128, 1)] == 0x7F).all()
    eq, es = ref.codes32(np.where(special, 1.0, t.double().cpu().numpy()), power)
    np.testing.assert_array_equal(s[~bad], es[~bad])
    np.testing.assert_array_equal(q[~np.repeat(bad, 128, 1)], eq[~np.repeat(bad, 128, 1)])


def test_quantize_row_stride(moe):
    """Rows that are a slice of wider ones; what lies between them is not read into a block."""
    rng = np.random.default_rng(4)
    wide = ref.bf16(rng.normal(0, 1, (37, 1024)))
    wide[:, :256] = 1e30
    wide[:, 656:] = 1e30
    t = ref.to_bf16_cuda(wide)
    q, s = moe.fp8_block_quantize_rows(t[:, 256:656])
    eq, es = ref.codes32(wide[:, 256:656])
    np.testing.assert_array_equal(host(s), es)
    np.testing.assert_array_equal(host(q), eq)
    q, s = moe.fp8_block_quantize_swiglu(t[:, 256:656])
    q2, s2 = moe.fp8_block_quantize_swiglu(t[:, 256:656].contiguous())
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("power", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 1024), (5, 200), (300, 1024), (64, 2048)])
def test_quantize_swiglu(moe, rows, cols, power):
    rng = np.random.default_rng(rows + cols)
    x = ref.bf16(rng.normal(0, 3, (rows, 2 * cols)))
    x[0, :4] = [100.0, -100.0, 0.0, -0.0]
    v = ref.silu_up(x)
    q, s = moe.fp8_block_quantize_swiglu(ref.to_bf16_cuda(x), scale_rule=moe.FP8_SCALE_POW2 if power else moe.FP8_SCALE_AMAX)
    q, s = host(q), host(s).astype(np.float64)
    amax = ref.block_amax(v)
    if power:
        assert np.all(s == 2.0 ** np.round(np.log2(s)))
        assert np.all(amax <= 448 * s * (1 + 2.0 ** -20)) and np.all(amax > 224 * s * (1 - 2.0 ** -20))
    else:
        assert np.all(np.abs(s - amax / 448) <= 2.0 ** -20 * amax / 448)
    got, step = ref.DECODE[q] * ref.expand(s, cols), ref.expand(s, cols)
    # half a step: 2^-4 of a normal code's value, 2^-10 among the subnormals
    assert np.all(np.abs(got - v) <= np.maximum(np.abs(v) / 16, step * 2.0 ** -10) * (1 + 2.0 ** -9))


# --- products ---------------------------------------------------------------------

def gemm_check(out, a, sa, w, sw, rows=None):
    """out against the 64-bit product of rows a (codes, scales) and weights w."""
    ra, rw = ref.real_rows(a, sa), ref.real_weights(w, sw)
    exact, mags = ra @ rw.T, np.abs(ra) @ np.abs(rw).T
    tol = (a.shape[1] + 8) * 2.0 ** -23 * mags
    got = out.double().cpu().numpy()
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(exact)
    assert np.all(np.abs(got - exact) <= tol), float(np.max(np.abs(got - exact) / np.maximum(tol, 1e-300)))


def operands(seed, M, N, K, experts=None):
    rng = np.random.default_rng(seed)
    lead = () if experts is None else (experts,)
    a, w = ref.random_codes(rng, M, K), ref.random_codes(rng, *lead, N, K)
    sa = np.exp2(rng.uniform(-12, -4, (M, ref.nb(K)))).astype(np.float32)
    sw = np.exp2(rng.uniform(-14, -8, lead + (ref.nb(N), ref.nb(K)))).astype(np.float32)
    return a, sa, w, sw


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 128, 128), (1, 7, 48), (2, 129, 144), (3, 256, 1024), (5, 64, 3584), (8, 320, 256), (9, 1000, 400),
    (16, 512, 2048), (17, 130, 272), (31, 384, 128), (33, 127, 640), (64, 256, 512), (65, 257, 528), (100, 2016, 1040),
    (127, 96, 384), (128, 128, 128), (129, 384, 1152), (200, 640, 256), (256, 256, 2048), (257, 520, 784), (300, 1536, 112),
    (513, 200, 640), (700, 1160, 896)])
def test_gemm(moe, M, N, K, dtype):
    a, sa, w, sw = operands(M + 31 * N + 7 * K, M, N, K)
    out = moe.fp8_block_gemm(dev(a), dev(sa), dev(w), dev(sw), out_dtype=dtype)
    assert out.dtype == dtype
    gemm_check(out, a, sa, w, sw)
    again = moe.fp8_block_gemm(dev(a), dev(sa), dev(w), dev(sw), out_dtype=dtype)
    assert torch.equal(out, again)
    assert moe.device_error() == 0


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_writes_its_output_alone(moe, M):
    """The values around an odd-sized output stay, and an output that starts off a 16-byte boundary is right."""
    N, K = 205, 272
    a, sa, w, sw = operands(M, M, N, K)
    for dt, pad in ((torch.bfloat16, 1), (torch.float32, 3)):
        buf = torch.full((M * N + 64,), 7.0, dtype=dt, device="cuda")
        out = buf[pad:pad + M * N].view(M, N)
        moe.fp8_block_gemm(dev(a), dev(sa), dev(w), dev(sw), out=out)
        gemm_check(out, a, sa, w, sw)
        assert (buf[:pad] == 7).all() and (buf[pad + M * N:] == 7).all()


def test_gemm_nan_stays_in_its_row_and_column(moe):
    M, N, K = 150, 140, 300 // 16 * 16
    a, sa, w, sw = operands(5, M, N, K)
    a[17, 200] = 0x7F
    w[33, 10] = 0xFF
    sa[80, 1] = np.nan
    out = host(moe.fp8_block_gemm(dev(a), dev(sa), dev(w), dev(sw), out_dtype=torch.float32))
    nan = np.zeros((M, N), bool)
    nan[17], nan[80], nan[:, 33] = True, True, True
    np.testing.assert_array_equal(np.isnan(out), nan)


@pytest.mark.parametrize("M", [3, 200])
def test_gemm_scale_blocks(moe, M):
    """Each scale applies to its own block: one block at a time scaled, the others by zero."""
    N, K = 300, 416
    a, sa, w, sw = operands(11, M, N, K)
    for b in range(ref.nb(K)):
        for c in range(ref.nb(N)):
            only_a, only_w = np.zeros_like(sa), np.zeros_like(sw)
            only_a[:, b], only_w[c, b] = sa[:, b], sw[c, b]
            out = moe.fp8_block_gemm(dev(a), dev(only_a), dev(w), dev(only_w), out_dtype=torch.float32)
            gemm_check(out, a, only_a, w, only_w)


def test_gemm_past_32_bits(moe):
    """An output of more than 2^31 values: rows from both ends against the 64-bit product."""
    M, N, K = 66000, 33000, 32
    rng = np.random.default_rng(3)
    a, w = ref.random_codes(rng, M, K), ref.random_codes(rng, N, K)
    sa, sw = np.full((M, 1), 0.01, np.float32), np.full((ref.nb(N), 1), 0.01, np.float32)
    out = moe.fp8_block_gemm(dev(a), dev(sa), dev(w), dev(sw))
    for r in (0, 1, 40000, M - 1):
        gemm_check(out[r:r + 1], a[r:r + 1], sa[r:r + 1], w, sw)


def test_gemm_other_stream(moe):
    a, sa, w, sw = operands(21, 90, 400, 512)
    t = [dev(v) for v in (a, sa, w, sw)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.empty(90, 400, dtype=torch.float32, device="cuda")
    moe.fp8_block_gemm(*t, out=out, stream=s)
    s.synchronize()
    gemm_check(out, a, sa, w, sw)


def test_gemm_in_a_graph(moe):
    """Captured and replayed over changed inputs, for few and many rows."""
    for M in (4, 300):
        a, sa, w, sw = operands(M, M, 512, 384)
        t = [dev(v) for v in (a, sa, w, sw)]
        out = torch.empty(M, 512, dtype=torch.float32, device="cuda")
        moe.fp8_block_gemm(*t, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.fp8_block_gemm(*t, out=out)
        b, sb, _, _ = operands(M + 1, M, 512, 384)
        t[0].copy_(dev(b))
        t[1].copy_(dev(sb))
        g.replay()
        gemm_check(out, b, sb, w, sw)


# --- the experts' products --------------------------------------------------------

def lists(ids, E):
    """offsets, pairs of [T, K] expert ids; ids outside [0, E) are in no list."""
    flat = ids.reshape(-1)
    offsets, pairs = [0], []
    for e in range(E):
        pairs += list(np.nonzero(flat == e)[0])
        offsets.append(len(pairs))
    pairs += [0] * (flat.size - len(pairs))
    return np.array(offsets, np.int32), np.array(pairs, np.int32)


def expert_check(moe, seed, T, topk, E, N, K, ids, in_rows, out_rows, dtype):
    rows = T if in_rows == moe.ROWS_TOKEN else T * topk
    a, sa, w, sw = operands(seed, rows, N, K, experts=E)
    offsets, pairs = lists(ids, E)
    out = torch.full((T * topk, N), 3.0, dtype=dtype, device="cuda")
    moe.expert_gemm(dev(a), dev(sa), dev(w), dev(sw), dev(offsets), dev(pairs), topk, in_rows=in_rows, out_rows=out_rows, out=out)
    written = np.zeros(T * topk, bool)
    for e in range(E):
        pos = np.arange(offsets[e], offsets[e + 1])
        if pos.size == 0:
            continue
        p = pairs[pos]
        src = {moe.ROWS_TOKEN: p // topk, moe.ROWS_LIST: pos, moe.ROWS_PAIR: p}[in_rows]
        dst = pos if out_rows == moe.ROWS_LIST else p
        written[dst] = True
        gemm_check(out[torch.from_numpy(dst.astype(np.int64)).cuda()], a[src], sa[src], w[e], sw[e])
    assert (out[torch.from_numpy(~written).cuda()] == 3.0).all()
    assert moe.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,topk,E,N,K", [
    (1, 1, 1, 16, 16), (1, 4, 8, 256, 384), (2, 2, 3, 130, 144), (8, 16, 64, 256, 512), (16, 3, 5, 200, 272),
    (37, 4, 16, 384, 256), (64, 8, 12, 136, 640), (130, 2, 2, 300, 400), (150, 4, 3, 257, 1040), (90, 16, 160, 128, 128)])
def test_expert_gemm(moe, T, topk, E, N, K, dtype):
    rng = np.random.default_rng(T * 7 + E)
    ids = np.stack([rng.permutation(E)[:topk] if topk <= E else rng.integers(0, E, topk) for _ in range(T)])
    expert_check(moe, T + E, T, topk, E, N, K, ids, moe.ROWS_TOKEN, moe.ROWS_PAIR, dtype)


@pytest.mark.parametrize("in_rows", ["ROWS_TOKEN", "ROWS_LIST", "ROWS_PAIR"])
@pytest.mark.parametrize("out_rows", ["ROWS_LIST", "ROWS_PAIR"])
@pytest.mark.parametrize("T", [6, 140])
def test_expert_rows(moe, in_rows, out_rows, T):
    rng = np.random.default_rng(1)
    ids = np.stack([rng.permutation(7)[:4] for _ in range(T)])
    expert_check(moe, 9, T, 4, 7, 264, 272, ids, getattr(moe, in_rows), getattr(moe, out_rows), torch.float32)


@pytest.mark.parametrize("case", ["one expert", "empty ends", "dropped", "all dropped", "skewed"])
def test_expert_loads(moe, case):
    """Experts without rows at both ends, every row at one expert, pairs in no list, one expert with most rows."""
    T, topk, E = 80, 4, 20
    rng = np.random.default_rng(2)
    ids = rng.integers(0, E, (T, topk))
    if case == "one expert":
        ids[:] = 13
    elif case == "empty ends":
        ids = rng.integers(5, 12, (T, topk))
    elif case == "dropped":
        ids[rng.random((T, topk)) < 0.3] = -1
    elif case == "all dropped":
        ids[:] = -1
    else:
        ids[rng.random((T, topk)) < 0.8] = 3
    expert_check(moe, 3, T, topk, E, 384, 400, ids, moe.ROWS_TOKEN, moe.ROWS_PAIR, torch.float32)


def test_expert_gemm_skips_bad_pairs(moe):
    """Pair codes and input rows out of range are skipped and reported; the other rows are right."""
    T, topk, E, N, K = 20, 2, 4, 140, 160
    rng = np.random.default_rng(8)
    ids = rng.integers(0, E, (T, topk))
    a, sa, w, sw = operands(1, T, N, K, experts=E)
    offsets, pairs = lists(ids, E)
    good = pairs.copy()
    pairs[3], pairs[10], pairs[30] = -1, T * topk, 2 ** 31 - 1
    out = torch.full((T * topk, N), 3.0, device="cuda")
    moe.expert_gemm(dev(a), dev(sa), dev(w), dev(sw), dev(offsets), dev(pairs), topk, out=out)
    assert moe.device_error() == moe.DEVERR_ROW_INDEX
    for e in range(E):
        for i in range(offsets[e], offsets[e + 1]):
            if i in (3, 10, 30):
                assert (out[good[i]] == 3.0).all()
            else:
                gemm_check(out[pairs[i]:pairs[i] + 1], a[pairs[i] // topk][None], sa[pairs[i] // topk][None], w[e], sw[e])
    # an input of fewer rows than the pairs name
    moe.expert_gemm(dev(a[:5]), dev(sa[:5]), dev(w), dev(sw), dev(offsets), dev(good), topk, out=out)
    assert moe.device_error() == moe.DEVERR_ROW_INDEX


def test_expert_gemm_skips_bad_pairs_of_long_lists(moe):
    """The same where lists are long (rows in list order are another path)."""
    T, topk, E, N, K = 200, 2, 2, 140, 160
    rng = np.random.default_rng(9)
    a, sa, w, sw = operands(1, T, N, K, experts=E)
    offsets, pairs = lists(rng.integers(0, E, (T, topk)), E)
    pairs[7], pairs[300] = -9, T * topk
    for in_rows, known in ((moe.ROWS_TOKEN, 150), (moe.ROWS_PAIR, 200), (moe.ROWS_LIST, 200)):
        out = torch.full((T * topk, N), 3.0, device="cuda")
        moe.expert_gemm(dev(a[:known]), dev(sa[:known]), dev(w), dev(sw), dev(offsets), dev(pairs), topk, in_rows=in_rows, out=out)
        assert moe.device_error() == moe.DEVERR_ROW_INDEX
        written = np.zeros(T * topk, bool)
        for e in range(E):
            pos = np.arange(offsets[e], offsets[e + 1])
            src = {moe.ROWS_TOKEN: pairs[pos] // topk, moe.ROWS_LIST: pos, moe.ROWS_PAIR: pairs[pos]}[in_rows]
            ok = (src >= 0) & (src < known) & (pairs[pos] >= 0) & (pairs[pos] < T * topk)
            written[pairs[pos][ok]] = True
            gemm_check(out[torch.from_numpy(pairs[pos][ok].astype(np.int64)).cuda()], a[src[ok]], sa[src[ok]], w[e], sw[e])
        assert (out[torch.from_numpy(~written).cuda()] == 3.0).all()


def test_expert_gemm_bad_offsets(moe):
    """Offsets past the list's ends, or descending, count as the nearest bound or as empty lists."""
    T, topk, E, N, K = 12, 2, 5, 64, 64
    a, sa, w, sw = operands(1, T, N, K, experts=E)
    pairs = np.arange(T * topk, dtype=np.int32)
    offsets = np.array([-5, 4, 4, 20, 10, 1000], np.int32)
    out = torch.full((T * topk, N), 3.0, device="cuda")
    moe.expert_gemm(dev(a), dev(sa), dev(w), dev(sw), dev(offsets), dev(pairs), topk, out=out)
    assert moe.device_error() == 0
    spans = [(0, 4), (4, 4), (4, 20), (20, 10), (10, 24)]
    for p in range(4):
        gemm_check(out[p:p + 1], a[p // 2][None], sa[p // 2][None], w[0], sw[0])
    for p in range(4, 10):
        gemm_check(out[p:p + 1], a[p // 2][None], sa[p // 2][None], w[2], sw[2])
    for p in range(20, 24):
        gemm_check(out[p:p + 1], a[p // 2][None], sa[p // 2][None], w[4], sw[4])
    assert spans[3][0] > spans[3][1]


@pytest.mark.parametrize("in_rows", ["ROWS_TOKEN", "ROWS_PAIR"])
@pytest.mark.parametrize("T,topk,E,N,K,copied", [(330, 2, 65, 1040, 4096, False), (700, 3, 65, 1040, 272, True), (350, 8, 65, 72, 400, True)])
def test_expert_rows_fetched_or_copied(moe, in_rows, T, topk, E, N, K, copied):
    """Lists of ten rows, fetched singly; of thirty for many columns, and of over forty: copied to list order first."""
    rng = np.random.default_rng(5)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(T)])
    rows = T if in_rows == "ROWS_TOKEN" else T * topk
    a, sa, _, _ = operands(4, rows, 8, K)
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randint(0, 0x78, (E, N, K), dtype=torch.uint8, device="cuda", generator=g)
    sw = torch.full((E, ref.nb(N), ref.nb(K)), 0.001, device="cuda")
    offsets, pairs = lists(ids, E)
    assert (moe.expert_gemm_workspace(T * topk, E, N, K, getattr(moe, in_rows)) > 0) == copied
    out = moe.expert_gemm(dev(a), dev(sa), w, sw, dev(offsets), dev(pairs), topk, in_rows=getattr(moe, in_rows), out_dtype=torch.float32)
    for e in (0, 31, 64):
        p = pairs[offsets[e]:offsets[e + 1]]
        src = p // topk if in_rows == "ROWS_TOKEN" else p
        gemm_check(out[torch.from_numpy(p.astype(np.int64)).cuda()], a[src], sa[src], host(w[e]), host(sw[e]))
    assert moe.device_error() == 0


def test_expert_weights_past_32_bits(moe):
    """Weights of more than 2^32 bytes: the last experts are reached."""
    E, N, K, T = 1100, 2048, 2048, 3
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randint(0, 0x78, (E, N, K), dtype=torch.uint8, device="cuda", generator=g)
    sw = torch.full((E, 16, 16), 0.001, device="cuda")
    rng = np.random.default_rng(0)
    a, sa = ref.random_codes(rng, T, K), np.full((T, 16), 0.01, np.float32)
    ids = np.array([[1099, 0], [1098, 1050], [1099, 1060]])
    offsets, pairs = lists(ids, E)
    out = moe.expert_gemm(dev(a), dev(sa), w, sw, dev(offsets), dev(pairs), 2, out_dtype=torch.float32)
    for t in range(T):
        for k in range(2):
            e = ids[t, k]
            gemm_check(out[2 * t + k:2 * t + k + 1], a[t:t + 1], sa[t:t + 1], host(w[e]), host(sw[e]))


# --- refusals ---------------------------------------------------------------------

def test_refusals(moe):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
    f = lambda *s: torch.zeros(*s, device="cuda")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        moe.fp8_block_quantize_rows(f(2, 128))
    with pytest.raises(ValueError):
        moe.fp8_block_quantize_rows(bf(128, 2).t())
    with pytest.raises(moe.MoeError):
        moe.fp8_block_quantize_rows(bf(2, 12))
    with pytest.raises(moe.MoeError):
        moe.fp8_block_quantize_rows(bf(2, 130)[:, :128])   # rows 260 bytes apart
    with pytest.raises(moe.MoeError):
        moe.fp8_block_quantize_rows(bf(2, 136)[:, 4:132])  # rows that start 8 bytes off
    with pytest.raises(moe.MoeError):
        moe.fp8_block_quantize_rows(bf(2, 128), scale_rule=2)
    with pytest.raises(ValueError):
        moe.fp8_block_quantize_rows(bf(2, 128), scales=f(2, 2))
    with pytest.raises(ValueError):
        moe.fp8_block_quantize_swiglu(bf(2, 129))
    with pytest.raises(moe.MoeError):
        moe.fp8_block_gemm(u8(2, 24), f(2, 1), u8(4, 24), f(1, 1))  # K % 16
    with pytest.raises(ValueError):
        moe.fp8_block_gemm(u8(2, 32), f(2, 1), u8(4, 48), f(1, 1))
    with pytest.raises(ValueError):
        moe.fp8_block_gemm(u8(2, 160), f(2, 1), u8(4, 160), f(1, 2))
    with pytest.raises(TypeError):
        moe.fp8_block_gemm(u8(2, 32), f(2, 1), u8(4, 32), f(1, 1), out_dtype=torch.float16)
    with pytest.raises(moe.MoeError):
        moe.fp8_block_gemm(u8(1, 40)[:, 8:].reshape(-1)[:32].view(1, 32), f(1, 1), u8(33 * 4)[4:4 + 128].view(4, 32), f(1, 1))
    args = lambda **k: dict(dict(a=u8(3, 32), a_scales=f(3, 1), w=u8(4, 8, 32), w_scales=f(4, 1, 1), offsets=i32(5), pairs=i32(6), topk=2), **k)
    with pytest.raises(ValueError):
        moe.expert_gemm(**args(offsets=i32(4)))
    with pytest.raises(moe.MoeError):
        moe.expert_gemm(**args(topk=0))
    with pytest.raises(moe.MoeError):
        moe.expert_gemm(**args(in_rows=3))
    with pytest.raises(moe.MoeError):
        moe.expert_gemm(**args(out_rows=moe.ROWS_TOKEN))
    # nothing to do
    assert moe.fp8_block_quantize_rows(bf(0, 128))[0].shape == (0, 128)
    assert moe.fp8_block_gemm(u8(0, 32), f(0, 1), u8(4, 32), f(1, 1)).shape == (0, 4)
    assert moe.expert_gemm(**args(pairs=i32(0))).shape == (0, 8)
    assert moe.device_error() == 0
