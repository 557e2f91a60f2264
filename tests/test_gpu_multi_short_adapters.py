"""Adapter gradients at ranks above 32 where adapters have from no token to a few blocks of 32: a workgroup's
first steps, which find their loads issued ahead of the loop, are then all there is."""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from _util import bits
from test_gpu_multi import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N,r,n,kind", [(20, 512, 384, 64, 3, "mixed"), (90, 288, 640, 40, 3, "mixed"),
                                            (300, 512, 384, 64, 40, "mixed"), (300, 96, 1024, 136, 6, "requests"),
                                            (33, 1024, 256, 256, 1, "one"), (1000, 320, 512, 100, 20, "requests")])
def test_gradients(gpu, T, K, N, r, n, kind):
    S, P, X, dY, A, B, di, U, res = run(gpu, T, K, N, r, n, kind)
    for name, x in (("bf16", X), ("ckpt", sra.ckpt8_encode(X))):
        for _ in range(5):  # the same bits however the loads happen to return
            again = sra.multi_lora_bwd(P, dY, x, U, A, B, di)
            for k in ("dA", "dB"):
                assert np.array_equal(bits(again[k]), bits(res[name][k])), (name, k)
