"""Host-side validation of the 8-bit block's calls: bad arguments are refused before any CUDA call
(no GPU needed)."""
import ctypes

import pytest

P = ctypes.c_void_p
A16 = P(256)  # a 16-byte aligned stand-in address; never dereferenced (validation fails first)
OFF = P(258)


@pytest.fixture(scope="module")
def lib():
    from latent_moe_decode_gb300 import build, load

    build.build()
    return load()


def test_route_grouped(lib):
    f = lambda T=4, E=64, K=8, scoring=0, G=8, KG=4, rule=1, logits=A16, ids=A16: lib.moe_topk_route_grouped(
        logits, None, T, E, K, scoring, G, KG, rule, 1, 1.0, ids, None, None, None)
    assert f(T=0) == 0
    for kw in (dict(T=-1), dict(E=0), dict(K=0), dict(G=0), dict(KG=0), dict(scoring=2), dict(rule=-1), dict(E=65), dict(KG=9),
               dict(K=33, E=64, KG=4), dict(K=9, KG=1), dict(logits=None), dict(ids=None)):
        assert f(**kw) == 1, kw
    assert f(E=4104) == 3
    assert f(K=33, KG=8) == 3
    assert f(E=4096, G=128, KG=64) == 3
    assert f(logits=OFF) == 2


def test_quantize(lib):
    for fn, width in ((lib.fp8_block_quantize_rows, 64), (lib.fp8_block_quantize_swiglu, 128)):
        f = lambda x=A16, ld=width, rows=4, cols=64, q=A16, s=A16, rule=0: fn(x, ld, rows, cols, q, s, rule, None)
        assert f(rows=0) == 0
        for kw in (dict(rows=-1), dict(cols=0), dict(cols=12), dict(ld=width - 8), dict(ld=width + 4), dict(rule=2), dict(rule=-1),
                   dict(x=None), dict(q=None), dict(s=None)):
            assert f(**kw) == 1, kw
        assert f(rows=2 ** 31 - 1) == 3
        assert f(x=P(264)) == 2 and f(q=P(260)) == 2 and f(s=OFF) == 2


def test_gemm(lib):
    f = lambda a=A16, sa=A16, w=A16, sw=A16, out=A16, dt=1, M=4, N=8, K=32: lib.fp8_block_gemm(a, sa, w, sw, out, dt, M, N, K, None)
    assert f(M=0) == 0 and f(N=0) == 0
    for kw in (dict(M=-1), dict(N=-1), dict(K=0), dict(K=24), dict(dt=2), dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(out=None)):
        assert f(**kw) == 1, kw
    assert f(a=P(264)) == 2 and f(w=P(264)) == 2 and f(sa=OFF) == 2 and f(sw=OFF) == 2 and f(out=P(257)) == 2 and f(out=OFF, dt=0) == 2


def test_expert_gemm(lib):
    f = lambda a=A16, rows=4, off=A16, pairs=A16, n=8, topk=2, i=0, o=2, out=A16, dt=1, E=4, N=8, K=32, ws=A16, wb=1 << 20: (
        lib.moe_expert_gemm(a, A16, rows, A16, A16, off, pairs, n, topk, i, o, out, dt, E, N, K, ws, wb, None))
    assert f(n=0) == 0 and f(N=0) == 0
    for kw in (dict(n=-1), dict(N=-1), dict(K=8), dict(K=40), dict(E=0), dict(topk=0), dict(rows=0), dict(i=3), dict(i=-1), dict(o=0), dict(o=3),
               dict(dt=2), dict(off=None), dict(pairs=None), dict(a=None), dict(out=None)):
        assert f(**kw) == 1, kw
    assert f(E=4097) == 3
    assert f(a=P(264)) == 2 and f(off=OFF) == 2 and f(pairs=OFF) == 2 and f(ws=P(264)) == 2
    # rows of long lists that are not in list order are copied there first
    need = lib.moe_expert_gemm_workspace
    assert need(8, 4, 8, 32, 0) == 0 and need(1000, 4, 8, 32, 1) == 0 and need(0, 4, 8, 32, 0) == 0 and need(1000, 4, 8, 8, 0) == 0
    assert need(1000, 4, 8, 160, 0) >= 1000 * 168 and need(1000, 4, 8, 160, 2) == need(1000, 4, 8, 160, 0)
    assert need(1000, 64, 128, 1024, 0) == 0 and need(1000, 64, 4096, 1024, 0) >= 1000 * 1056  # (few weights; many)
    assert f(n=1000, wb=need(1000, 4, 8, 32, 0) - 1) == 4 and f(n=1000, ws=None) == 4


def test_block_norm(lib):
    f = lambda y=A16, ld=64, r=A16, dt=1, post=A16, gate=None, kind=0, nxt=A16, eps=1e-6, T=4, H=64, h=A16, n=A16, q=None, s=None: (
        lib.moe_block_norm(y, ld, r, dt, post, gate, kind, nxt, 1.0, eps, T, H, h, n, q, s, None))
    assert f(T=0) == 0
    for kw in (dict(T=-1), dict(H=0), dict(H=60), dict(ld=56), dict(ld=68), dict(eps=-1.0), dict(eps=float("nan")), dict(dt=2), dict(kind=4, gate=A16),
               dict(kind=1), dict(gate=A16), dict(q=A16), dict(s=A16), dict(y=None), dict(r=None), dict(nxt=None), dict(h=None)):
        assert f(**kw) == 1, kw
    assert f(H=16392, ld=16392) == 3
    assert f(y=P(264)) == 2 and f(n=P(264)) == 2 and f(gate=P(257), kind=1) == 2 and f(gate=P(258), kind=2) == 2 and f(q=P(260), s=A16) == 2
