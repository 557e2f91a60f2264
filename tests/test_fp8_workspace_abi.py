"""The size of the 8-bit product's workspace does not depend on the tuning knob of its tiles (no GPU, no launch)."""
import pytest

import sparse_rank_adapter_amd as sra


@pytest.mark.parametrize("M,N,K", [(64, 64, 8192), (40, 128, 4096), (100, 64, 1024), (200, 300, 20480)])
@pytest.mark.parametrize("tile", [64, 128, 132, 256])
def test_knob_leaves_the_workspace(M, N, K, tile):
    sra.fp8_matmul_workspace.cache_clear()
    with sra.tuned(fp8_tile=tile):
        tuned = sra.fp8_matmul_workspace(M, N, K)
    sra.fp8_matmul_workspace.cache_clear()
    assert sra.fp8_matmul_workspace(M, N, K) == tuned > 0
