"""The 8-bit product of few rows by few rows over a long reduction splits it over the chip, and others still need no
workspace (no GPU, no launch)."""
import pytest

import sparse_rank_adapter_amd as sra


@pytest.mark.parametrize("M,N,K", [(32, 64, 1 << 20), (1, 64, 1 << 20), (1, 1, 1 << 22), (16, 256, 1 << 17), (32, 2048, 16384), (32, 16, 36864)])
def test_split(M, N, K):
    assert sra.fp8_matmul_workspace(M, N, K) >= 2 * M * N * 4
    # as many parts as with a row more than the streaming kernel takes
    assert sra.fp8_matmul_workspace(M, N, K) * 33 == sra.fp8_matmul_workspace(33, N, K) * M


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (16, 64, 1024), (32, 1024, 4096), (1, 4096, 4096), (16, 36864, 9216), (32, 20480, 5120),
                                   (8, 8192, 1 << 20), (1, 5120, 20480), (17, 1000, 0)])
def test_streamed(M, N, K):
    assert sra.fp8_matmul_workspace(M, N, K) == 0
