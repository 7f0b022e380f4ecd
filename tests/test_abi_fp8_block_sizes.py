"""Host-side sizes of the 8-bit block's calls at their ends: none at all, and the most that an index
holds (no GPU needed: refused, or nothing to do, before any CUDA call)."""
import ctypes

import pytest

A16 = ctypes.c_void_p(256)  # a 16-byte aligned stand-in address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from latent_moe_decode_gb300 import build, load

    build.build()
    return load()


def expert_gemm(lib, rows, n, ws=None, wb=0, E=4, N=8, K=32):
    return lib.moe_expert_gemm(A16, A16, rows, A16, A16, A16, A16, n, 2, 0, 2, A16, 1, E, N, K, ws, wb, None)


def test_expert_gemm_of_an_empty_batch(lib):
    assert expert_gemm(lib, 0, 0) == 0
    assert expert_gemm(lib, 0, 1) == 1 and expert_gemm(lib, -1, 0) == 1 and expert_gemm(lib, -1, 8) == 1


def test_expert_gemm_of_more_pairs_than_its_indices_hold(lib):
    """The list copy's loop steps past the last pair by what its warps take at a time."""
    for n in (2 ** 31 - 1, 2 ** 31 - 2 ** 16):
        assert expert_gemm(lib, 1, n, A16, 2 ** 62) == 3
