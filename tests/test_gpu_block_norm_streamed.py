"""The streamed block norm (more rows than SMs): rings that go round more than once, every gate, with and
without the post norm, with and without codes and n, h over the residual whose next rows are already on their
way, strided y, and rows too long for one fragment a thread. Tolerances as in test_gpu_block_norm."""
import numpy as np
import pytest
import torch

import block_reference as ref
from gpu_helpers import dev
from test_gpu_block_norm import case, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("T,H", [(3000, 264), (900, 4104), (700, 8200)])
def test_streamed(moe, T, H, gate, post, f32):
    check(moe, *case(T + H, T, H, f32, gate, post), alpha=0.7, eps=1e-6, f32=f32, quantize=True)


@pytest.mark.parametrize("T,H,gate", [(3000, 7168, "full"), (160, 8192, "channel"), (153, 16384, "none"), (400, 16384, "full"), (20000, 8, "token")])
def test_streamed_sizes(moe, T, H, gate):
    check(moe, *case(T, T, H, True, gate, True), alpha=-1.25, eps=1e-5, f32=True, quantize=False)


@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_streamed_in_place_with_strided_rows(moe, gate, post, f32):
    T, H = 2500, 1032
    y, r, p, g, nxt = case(11, T, H, f32, gate, post)
    expect = run(moe, y, r, p, g, nxt, 0.7, 1e-6, f32, True)
    t = ref.to_bf16_cuda
    wide = torch.full((T, 2 * H), 1e30, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + H] = t(y)
    residual = dev(r.astype(np.float32)) if f32 else t(r)
    got = moe.block_norm(wide[:, 8:8 + H], residual, t(nxt), post_weight=None if p is None else t(p), gate=None if g is None else t(g), alpha=0.7,
                         eps=1e-6, h=residual, quantize=True)
    assert got[0] is residual
    for u, v in zip(expect, got):
        assert torch.equal(u, v)
    again = run(moe, y, r, p, g, nxt, 0.7, 1e-6, f32, False)
    assert torch.equal(again[0], expect[0]) and torch.equal(again[1], expect[1])
    assert moe.device_error() == 0
