"""A workspace that the caller passes: any CUDA tensor of contiguous bytes enough; anything else is refused
before a launch."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def calls(moe):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
    f = lambda *s: torch.zeros(*s, device="cuda")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    pairs = torch.arange(200, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    T, E, L = 8, 64, 64
    return {
        "expert_gemm": (moe.expert_gemm_workspace(200, 1, 64, 128), lambda ws: moe.expert_gemm(
            u8(100, 128), f(100, 1), u8(1, 64, 128), f(1, 1, 1), offsets, pairs, 2, workspace=ws)),
        "router_logits": (moe.router_logits_workspace(T, 512, E), lambda ws: moe.router_logits(bf(T, 512), bf(E, 512), workspace=ws)),
        "front_projection": (moe.front_projection_workspace(T, 512, E, L), lambda ws: moe.front_projection(bf(T, 512), bf(E, 512), bf(L, 512), workspace=ws)),
        "build_routing_lists": (moe.build_routing_lists_workspace(T, 8, E), lambda ws: moe.build_routing_lists(i32(T, 8), E, workspace=ws)),
        "route_finalize": (moe.route_finalize_workspace(T, 512, E, 8), lambda ws: moe.route_finalize(
            bf(T, 512), bf(E, 512), None, bf(T, L), bf(T * 8, L), 8, True, 1.0, f(T, E), i32(T, 8), f(T, 8), bf(T, 8), i32(E + 1), i32(T * 8), u8(T, L),
            u8(T, L // 32), bf(T, L), workspace=ws)),
    }


def test_workspaces(moe):
    refused = 0
    for name, (need, call) in calls(moe).items():
        size = max(need, 64)
        for bad, error in ((torch.zeros(size, dtype=torch.uint8), ValueError), (torch.zeros(2 * size, dtype=torch.uint8, device="cuda")[::2], ValueError),
                           (b"0" * size, TypeError)):
            with pytest.raises(error, match="workspace"):
                call(bad)
        if need:
            refused += 1
            with pytest.raises(moe.MoeError):
                call(torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))
        call(torch.zeros(size // 4 + 1, device="cuda"))  # (of another type)
    assert refused >= 1  # expert_gemm's lists here are copied
    torch.cuda.synchronize()
    assert moe.device_error() == 0
