"""One mixture-of-experts block in 8-bit floating point, from the residual stream back to it.

    python examples/moe_block.py [tokens]

The block takes the residual stream and the preceding block's output, and runs

    norm after that block, residual, norm before this one, codes   block_norm
    router logits                                                  router_logits
    the choice of experts and their weights                        topk_route_grouped
    lists by expert                                                build_routing_lists
    latent rows (down projection), their codes                     fp8_block_gemm, fp8_block_quantize_rows
    the experts' gate and up product                               expert_gemm (token rows in, list rows out)
    silu(gate) * up and its codes                                  fp8_block_quantize_swiglu
    the experts' down product                                      expert_gemm (list rows in, pair rows out)
    the weighted sum of a token's experts                          finalize
    back to the hidden size (up projection)                        fp8_block_quantize_rows, fp8_block_gemm

Every buffer is allocated once, so a step can be captured in a CUDA graph.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import latent_moe_decode_gb300 as moe  # noqa: E402


def block_weights(w):
    """(E4M3 codes uint8, FP32 scales per 128 x 128 block) of weights [..., N, K]: once, at load."""
    n, k = w.shape[-2:]
    nb, kb = -(-n // 128), -(-k // 128)
    p = torch.nn.functional.pad(w.float(), (0, kb * 128 - k, 0, nb * 128 - n))
    b = p.view(*w.shape[:-2], nb, 128, kb, 128)
    scale = (b.abs().amax((-3, -1)) / 448.0).clamp_min(2.0 ** -100)
    q = (b / scale[..., :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(*w.shape[:-2], nb * 128, kb * 128)[..., :n, :k].contiguous(), scale.contiguous()


class MoeBlock:
    """Sizes: T tokens, hidden H, latent L, E experts of F columns, K of them per token, in n_group
    groups of which topk_group are kept."""

    def __init__(self, T, H, L, F, E, K, n_group=1, topk_group=1, scale=2.5, alpha=1.0, eps=1e-6, seed=0, device="cuda"):
        self.T, self.H, self.L, self.F, self.E, self.K = T, H, L, F, E, K
        self.n_group, self.topk_group, self.scale, self.alpha, self.eps = n_group, topk_group, scale, alpha, eps
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)
        bf = lambda t: t.to(torch.bfloat16)
        self.post_norm, self.next_norm = bf(1 + 0.1 * rand(H)), bf(1 + 0.1 * rand(H))
        self.gate = bf(0.02 * rand(E, H))
        self.bias = 0.01 * rand(E)
        self.w_down, self.s_down = block_weights(rand(L, H) / H ** 0.5)
        self.w_up, self.s_up = block_weights(rand(H, L) / L ** 0.5)
        experts = lambda n, k: [torch.stack(v) for v in zip(*(block_weights(rand(n, k) / k ** 0.5) for _ in range(E)))]
        self.w_gu, self.s_gu = experts(2 * F, L)
        self.w_dn, self.s_dn = experts(L, F)
        # buffers
        u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=device)
        f32 = lambda *s: torch.empty(*s, dtype=torch.float32, device=device)
        b16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=device)
        i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device=device)
        nb = lambda n: -(-n // 128)
        P = T * K
        self.h, self.n, self.q, self.s = f32(T, H), b16(T, H), u8(T, H), f32(T, nb(H))
        self.logits, self.router_ws = f32(T, E), u8(max(1, moe.router_logits_workspace(T, H, E)))
        self.ids, self.weights, self.weights_bf16 = i32(T, K), f32(T, K), b16(T, K)
        self.offsets, self.pairs = i32(E + 1), i32(P)
        self.lists_ws = u8(max(1, moe.build_routing_lists_workspace(T, K, E)))
        self.latent, self.lq, self.ls = b16(T, L), u8(T, L), f32(T, nb(L))
        self.gu, self.aq, self.as_ = b16(P, 2 * F), u8(P, F), f32(P, nb(F))
        self.gu_ws = u8(max(1, moe.expert_gemm_workspace(P, E, 2 * F, L)))
        self.rows, self.routed, self.rq, self.rs = b16(P, L), b16(T, L), u8(T, L), f32(T, nb(L))
        self.y = b16(T, H)

    def run(self, y, residual):
        """(this block's output BF16 [T, H], the residual stream FP32 [T, H]) from the preceding block's
        output y (BF16) and the stream before it (FP32)."""
        moe.block_norm(y, residual, self.next_norm, post_weight=self.post_norm, alpha=self.alpha, eps=self.eps, h=self.h, n=self.n,
                       quantize=True, q=self.q, scales=self.s)
        moe.router_logits(self.n, self.gate, out=self.logits, workspace=self.router_ws)
        moe.topk_route_grouped(self.logits, self.bias, self.K, self.n_group, self.topk_group, scale=self.scale, ids=self.ids,
                               weights=self.weights, weights_bf16=self.weights_bf16)
        moe.build_routing_lists(self.ids, self.E, offsets=self.offsets, pairs=self.pairs, workspace=self.lists_ws)
        moe.fp8_block_gemm(self.q, self.s, self.w_down, self.s_down, out=self.latent)
        moe.fp8_block_quantize_rows(self.latent, q=self.lq, scales=self.ls)
        moe.expert_gemm(self.lq, self.ls, self.w_gu, self.s_gu, self.offsets, self.pairs, self.K, in_rows=moe.ROWS_TOKEN,
                        out_rows=moe.ROWS_LIST, out=self.gu, workspace=self.gu_ws)
        moe.fp8_block_quantize_swiglu(self.gu, q=self.aq, scales=self.as_)
        moe.expert_gemm(self.aq, self.as_, self.w_dn, self.s_dn, self.offsets, self.pairs, self.K, in_rows=moe.ROWS_LIST,
                        out_rows=moe.ROWS_PAIR, out=self.rows)
        moe.finalize(self.rows, self.weights_bf16, self.T, self.K, out=self.routed)
        moe.fp8_block_quantize_rows(self.routed, q=self.rq, scales=self.rs)
        moe.fp8_block_gemm(self.rq, self.rs, self.w_up, self.s_up, out=self.y)
        return self.y, self.h


def main():
    T = int(sys.argv[1]) if len(sys.argv) > 1 else 64
    block = MoeBlock(T, H=7168, L=3584, F=1024, E=256, K=8, n_group=8, topk_group=4)
    y = torch.randn(T, block.H, device="cuda").to(torch.bfloat16)
    residual = torch.randn(T, block.H, device="cuda")
    block.run(y, residual)  # (loads the kernels before the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, stream = block.run(y, residual)
    for _ in range(3):
        graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert moe.device_error() == 0 and torch.isfinite(out).all() and torch.isfinite(stream).all()
    us = start.elapsed_time(end) * 1e3 / 20
    print(f"{T} tokens, hidden {block.H}, latent {block.L}, {block.K} of {block.E} experts of {block.F}: {us:.1f} us a block, {T / us:.3f} M tokens/s")


if __name__ == "__main__":
    main()
