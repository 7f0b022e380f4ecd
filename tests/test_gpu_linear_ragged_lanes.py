"""The BF16 products where a warp's lanes part: columns that end inside a warp of weights, with the K of one tile
left whole or split, one chunk of rows or several; the column sums of rows that end inside a warp."""
import pytest
import torch

from test_gpu_linear import BF, F32, check_gated, check_linear, check_linear_backward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 5, 16, 31, 48, 65, 100, 176])
@pytest.mark.parametrize("n", [1, 31, 33, 127, 129, 161, 259])
def test_columns_that_end_inside_a_warp(moe, t, n):
    for k in (40, 64, 520):  # (one block of K has nothing to split)
        check_linear(moe, t, n, k, "silu", F32, F32, F32, pre=True)
        check_linear(moe, t, n, k, "gelu", BF, BF, BF, pad=1)
        check_gated(moe, t, n, k)


@pytest.mark.parametrize("t", [1, 2, 5, 31, 33, 130, 1025, 2049])
def test_sums_of_rows_that_end_inside_a_warp(moe, t):
    for n in (3, 8, 72, 129):
        check_linear_backward(moe, t, n, 16, "silu")
        check_linear_backward(moe, t, n, 16, odd_dout=True)
