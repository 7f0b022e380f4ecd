"""The BF16 products' calls at the same time: on two streams that are seen to overlap, from two threads, in two
graphs; and their workspaces."""
import threading

import pytest
import torch

from test_gpu_linear import BF, F32, rand

pytestmark = pytest.mark.gpu

# (both kernels, K whole and split over clusters, tiles of few and of all TMEM columns)
SIZES = [(1, 7168, 2048), (3, 3584, 1024), (64, 1024, 2048), (97, 4096, 1024), (176, 2018, 4096), (250, 2048, 512), (700, 1024, 1024)]


def data(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(rand(g, t, k), rand(g, n, k, scale=k ** -0.5), rand(g, t, n), rand(g, t, n)) for t, n, k in SIZES]


def calls(moe, v, s=None):
    """One call after another, so that two streams' can be dealt out in turn."""
    for x, w, d, p in v:
        f = w.shape[0] // 2
        yield (moe.bf16_linear(x, w, out_dtype=F32, stream=s)[0],)
        yield moe.bf16_gated_linear(x, w, want_pre=True, stream=s)
        yield moe.bf16_linear_backward(d, x, w, p, moe.ACT_GELU, want_dbias=True, stream=s)
        yield moe.bf16_gated_linear_backward(d[:, :f], x, w, p, stream=s)


def check(got, expect):
    for a, b in zip(got, expect, strict=True):
        assert all(torch.equal(u, v) if v is not None else u is None for u, v in zip(a, b, strict=True))


def overlap(marks):
    """Whether both intervals had begun before either ended."""
    (a0, a1), (b0, b1) = marks
    return a0.elapsed_time(b1) > 0 and b0.elapsed_time(a1) > 0


def test_two_streams_that_overlap(moe):
    """Both held back until all calls are queued, then let go at once."""
    sides = [data(1), data(2)]
    expect = [list(calls(moe, v)) for v in sides]
    torch.cuda.synchronize()
    streams, hold = [torch.cuda.Stream() for _ in range(2)], torch.cuda.Stream()
    for _ in range(5):
        go, marks = torch.cuda.Event(), [[torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in range(2)]
        with torch.cuda.stream(hold):
            torch.cuda._sleep(60_000_000)  # (some 30 ms; the calls are queued in 5)
            go.record()
        for s, (start, _) in zip(streams, marks):
            s.wait_event(go)
            start.record(s)
        got = [[], []]
        for a, b in zip(*(calls(moe, v, s) for v, s in zip(sides, streams)), strict=True):
            got[0].append(a)
            got[1].append(b)
        assert not go.query()  # nothing has run yet
        for s, (_, end) in zip(streams, marks):
            end.record(s)
        torch.cuda.synchronize()
        assert overlap(marks)
        for a, b in zip(got, expect):
            check(a, b)
    assert moe.device_error() == 0


def test_two_graphs_that_overlap(moe):
    sides = [data(3), data(4)]
    expect = [list(calls(moe, v)) for v in sides]
    torch.cuda.synchronize()
    graphs, got = [], []
    for v in sides:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(list(calls(moe, v)))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    seen = 0
    for _ in range(20):
        for r in got:
            for v in r:
                for o in v:
                    o.zero_()
        torch.cuda.synchronize()
        marks = [[torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in range(2)]
        for s, g, (start, end) in zip(streams, graphs, marks):
            with torch.cuda.stream(s):
                start.record()
                for _ in range(5):
                    g.replay()
                end.record()
        torch.cuda.synchronize()
        seen += overlap(marks)
        for a, b in zip(got, expect):
            check(a, b)
    assert seen > 0
    assert moe.device_error() == 0


def test_two_threads(moe):
    """Each with sizes of its own (and its own memory of their plans), again and again."""
    sides = [data(5), list(reversed(data(6)))]
    expect = [list(calls(moe, v)) for v in sides]
    torch.cuda.synchronize()
    errors, device = [], torch.cuda.current_device()

    def body(v, e):
        try:
            torch.cuda.set_device(device)
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got = list(calls(moe, v))
                s.synchronize()
                check(got, e)
        except Exception as error:  # noqa: BLE001 -- reported below
            errors.append(error)

    threads = [threading.Thread(target=body, args=a) for a in zip(sides, expect)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert moe.device_error() == 0


def test_workspaces(moe):
    """A workspace that the caller passes: any CUDA tensor of contiguous bytes enough, of which nothing past the bytes
    asked for is touched; anything else is refused before a launch."""
    g = torch.Generator(device="cuda").manual_seed(7)
    t, n, k = 37, 130, 72
    x, w, d, p = rand(g, t, k), rand(g, n, k), rand(g, t, n), rand(g, t, n)
    for need, call in ((moe.bf16_linear_backward_workspace(t, n), lambda ws: moe.bf16_linear_backward(d, x, w, p, moe.ACT_SILU, want_dbias=True, workspace=ws)),
                       (moe.bf16_gated_linear_backward_workspace(t, n // 2), lambda ws: moe.bf16_gated_linear_backward(d[:, :n // 2], x, w, p, workspace=ws))):
        assert need == t * 192 * 2
        expect = call(None)
        for bad, error in ((torch.zeros(need, dtype=torch.uint8), ValueError), (torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2], ValueError),
                           (b"0" * need, TypeError)):
            with pytest.raises(error, match="workspace"):
                call(bad)
        with pytest.raises(moe.MoeError) as short:
            call(torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))
        assert short.value.status == moe.ERR_WORKSPACE
        ws = torch.full((need + 256,), 0x55, dtype=torch.uint8, device="cuda")
        check([call(ws[:need])], [expect])
        assert (ws[need:] == 0x55).all()
        check([call(torch.full((need // 4,), float("nan"), device="cuda"))], [expect])  # (of another type, and what it holds does not matter)
    # without an activation dout itself serves: no workspace, and one that is too small is not looked at
    expect = moe.bf16_linear_backward(d[:, :128].contiguous(), x, w[:128])
    check([moe.bf16_linear_backward(d[:, :128].contiguous(), x, w[:128], workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))], [expect])
    torch.cuda.synchronize()
    assert moe.device_error() == 0
