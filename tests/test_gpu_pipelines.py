"""The persistent kernels where a CTA (or pair) takes several tiles, so that every ring of stages and
accumulators goes round and its parities turn: even and odd counts of K blocks, one block, a partial last
one. Tolerances as for the products."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev
from test_gpu_fp8_block import expert_check, gemm_check, operands

pytestmark = pytest.mark.gpu


# 100 and more tiles of 256 x 256 for 76 pairs; 313 and more of 128 weight rows for 152 CTAs
@pytest.mark.parametrize("M,N,K", [
    (2560, 2560, 128), (2560, 2560, 384), (2500, 2599, 640), (2560, 2500, 1024), (5000, 2600, 400), (2304, 5200, 1168),
    (10, 40000, 272), (20, 40000, 640), (64, 40001, 384), (64, 60000, 128), (33, 20000, 1664)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dense(moe, M, N, K, dtype):
    a, sa, w, sw = operands(M + N + K, M, N, K)
    t = [dev(v) for v in (a, sa, w, sw)]
    out = moe.fp8_block_gemm(*t, out_dtype=dtype)
    gemm_check(out, a, sa, w, sw)
    for _ in range(20):  # calls in a row, each while the last one ends
        again = moe.fp8_block_gemm(*t, out_dtype=dtype)
    assert torch.equal(out, again)
    assert moe.device_error() == 0


@pytest.mark.parametrize("in_rows", ["ROWS_TOKEN", "ROWS_LIST"])
@pytest.mark.parametrize("T,topk,E,N,K", [
    (3000, 2, 6, 1040, 640), (3000, 2, 6, 1040, 272), (1000, 3, 5, 2600, 128),  # 256 rows a tile
    (1625, 2, 65, 1040, 272), (1625, 2, 65, 1040, 512), (1625, 2, 65, 1040, 112),  # 64
    (650, 2, 65, 1040, 272), (650, 2, 65, 1040, 640),                              # 32
    (260, 2, 65, 1040, 384), (260, 2, 65, 1040, 128)])                             # 16
def test_experts(moe, T, topk, E, N, K, in_rows):
    rng = np.random.default_rng(T + K)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(T)])
    expert_check(moe, T + E, T, topk, E, N, K, ids, getattr(moe, in_rows), moe.ROWS_PAIR, torch.float32)
