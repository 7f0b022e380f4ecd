"""Calls on a stream that is not the current one, whose results and scratch the binding allocates: while the
launch waits on its stream, the current stream takes and fills memory of the same sizes. Neither
side may touch the other's."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def operands():
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    codes = lambda *s: torch.randint(0, 0x78, s, generator=g, device="cuda", dtype=torch.uint8)
    bf = lambda *s: rand(*s).to(torch.bfloat16)
    T, topk, E = 2000, 4, 8
    ids = torch.randint(0, E, (T, topk), generator=g, device="cuda", dtype=torch.int32)
    return dict(T=T, topk=topk, E=E, ids=ids, x=bf(T, 1024), w_router=bf(256, 1024), w_down=bf(384, 1024), logits=rand(T, 256), bias=0.1 * rand(256),
                a=codes(T, 1024), sa=rand(T, 8).abs(), w=codes(E, 256, 1024), sw=rand(E, 2, 8).abs(), residual=rand(T, 1024),
                gate_up=bf(T, 512), next=bf(1024), weights=rand(T, topk).abs(), rows=bf(T * topk, 256))


def calls(moe, o):
    offsets, pairs = moe.build_routing_lists(o["ids"], o["E"])
    assert moe.expert_gemm_workspace(o["T"] * o["topk"], o["E"], 256, 1024) > 0
    return dict(
        expert_gemm=lambda s: moe.expert_gemm(o["a"], o["sa"], o["w"], o["sw"], offsets, pairs, o["topk"], stream=s),
        fp8_block_gemm=lambda s: moe.fp8_block_gemm(o["a"], o["sa"], o["w"][0], o["sw"][0], stream=s),
        fp8_block_quantize_rows=lambda s: moe.fp8_block_quantize_rows(o["x"], stream=s),
        fp8_block_quantize_swiglu=lambda s: moe.fp8_block_quantize_swiglu(o["gate_up"], stream=s),
        block_norm=lambda s: moe.block_norm(o["x"], o["residual"], o["next"], quantize=True, stream=s),
        topk_route_grouped=lambda s: moe.topk_route_grouped(o["logits"], o["bias"], 8, n_group=8, topk_group=4, stream=s),
        topk_route=lambda s: moe.topk_route(o["logits"], o["bias"], 8, stream=s),
        router_logits=lambda s: moe.router_logits(o["x"], o["w_router"], stream=s),
        front_projection=lambda s: moe.front_projection(o["x"], o["w_router"], o["w_down"], stream=s),
        build_routing_lists=lambda s: moe.build_routing_lists(o["ids"], o["E"], stream=s),
        mxfp8_quantize_rows=lambda s: moe.mxfp8_quantize_rows(o["x"], stream=s),
        finalize=lambda s: moe.finalize(o["rows"], o["weights"], o["T"], o["topk"], stream=s),
    )


def test_results_and_scratch_of_another_stream(moe):
    o = operands()
    for name, call in calls(moe, o).items():
        expect = call(None)
        expect = [t.clone() for t in (expect if isinstance(expect, tuple) else (expect,))]
        sizes = {t.numel() * t.element_size() for t in expect} | {o["T"] * o["topk"] * 1056, moe.router_logits_workspace(o["T"], 1024, 256),
                                                                  moe.build_routing_lists_workspace(o["T"], o["topk"], o["E"])}
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)  # about 10 ms
        got = call(s)
        call(s)  # (its results are dropped at once)
        theirs = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes if n for _ in range(4)]
        s.synchronize()
        for u, v in zip(expect, got if isinstance(got, tuple) else (got,)):
            assert torch.equal(u, v), name
        assert all(bool((t == 0x55).all()) for t in theirs), name
        del theirs
    assert moe.device_error() == 0


def test_results_stay_while_the_current_stream_reads_them(moe):
    """A result made on another stream, dropped while the current stream still reads it."""
    o = operands()
    expect = moe.fp8_block_quantize_rows(o["x"])[0].clone()
    zeros = torch.zeros_like(o["x"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q = moe.fp8_block_quantize_rows(o["x"], stream=s)[0]
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(20_000_000)
    copy = q.clone()
    del q
    for _ in range(4):
        moe.fp8_block_quantize_rows(zeros, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(copy, expect)


def test_another_stream_in_a_captured_fork(moe):
    """A call on a side stream of a capture, its results and scratch allocated there, replayed over changed rows."""
    o = operands()
    offsets, pairs = moe.build_routing_lists(o["ids"], o["E"])
    args = (o["a"], o["sa"], o["w"], o["sw"], offsets, pairs, o["topk"])
    moe.expert_gemm(*args)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        out = moe.expert_gemm(*args, stream=side)
        codes = moe.fp8_block_quantize_rows(o["x"])  # (beside it)
        main.wait_stream(side)
    for _ in range(3):
        o["a"].copy_(o["a"].roll(1, 0))
        out.zero_()
        graph.replay()
        assert torch.equal(out, moe.expert_gemm(*args))
    assert torch.equal(codes[0], moe.fp8_block_quantize_rows(o["x"])[0])
    assert moe.device_error() == 0
