"""Malformed lists where the rows are copied to list order first: offsets that descend, or start past
0, give the rows that the fetched path gives, and what no list holds is neither read nor reported.
Tolerances as for the products."""
import numpy as np
import pytest
import torch

import block_reference as ref
from gpu_helpers import dev
from test_gpu_fp8_block import gemm_check, operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_rows", ["ROWS_TOKEN", "ROWS_PAIR"])
@pytest.mark.parametrize("offsets", [
    [20, 200, 400, 350, 60, 120],              # 256 rows a tile; lists end past the last offset, and descend
    [20, 200, 400, 350, 350, 60, 60, 120],     # 64 rows a tile
    [900, 20, 200, 200, 390, -3],              # the first list empty, the last offset 0
    [380, 400, 10, 150, 150, 150, 100, 130]])  # lists that start below the first offset
def test_descending_offsets(moe, offsets, in_rows):
    T, topk, N, K = 200, 2, 140, 272
    E, P = len(offsets) - 1, T * topk
    rows = T if in_rows == "ROWS_TOKEN" else P
    a, sa, w, sw = operands(7, rows, N, K, experts=E)
    pairs = np.random.default_rng(3).permutation(P).astype(np.int32)
    ends = np.clip(offsets, 0, P)
    owner = np.full(P, -1)
    for e in range(E):
        for i in range(ends[e], ends[e + 1]):
            owner[i] = e if owner[i] == -1 else -2  # (in two lists: either's)
    names = pairs.copy()
    names[owner == -1] = -7  # (in no list)
    need = moe.expert_gemm_workspace(P, E, N, K, getattr(moe, in_rows))
    assert need > 0
    out = torch.full((P, N), 3.0, device="cuda")
    moe.expert_gemm(dev(a), dev(sa), dev(w), dev(sw), dev(np.array(offsets, np.int32)), dev(names), topk, in_rows=getattr(moe, in_rows), out=out,
                    workspace=torch.full((need,), 0x7F, dtype=torch.uint8, device="cuda"))
    assert moe.device_error() == 0
    for e in range(E):
        p = pairs[owner == e]
        if p.size:
            src = p // topk if in_rows == "ROWS_TOKEN" else p
            gemm_check(out[torch.from_numpy(p.astype(np.int64)).cuda()], a[src], sa[src], w[e], sw[e])
    assert (out[torch.from_numpy(pairs[owner == -1].astype(np.int64)).cuda()] == 3.0).all()


def test_empty_batch(moe):
    """No tokens: an output of no rows, by every row mode."""
    f = lambda *s: torch.zeros(*s, device="cuda")
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    for rows in (moe.ROWS_TOKEN, moe.ROWS_LIST, moe.ROWS_PAIR):
        assert moe.expert_gemm(u8(0, 32), f(0, 1), u8(4, 8, 32), f(4, 1, 1), i32(5), i32(0), 2, in_rows=rows).shape == (0, 8)
