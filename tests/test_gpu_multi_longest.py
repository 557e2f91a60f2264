"""The longest batch of the many-adapter forward, 2^26 - 1 tokens, at a rank of two column tiles with more
adapters than a launch has room to take side by side.  Most tokens are zero; tolerances as in test_gpu_multi."""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import multi as om
from _util import f64
from test_gpu_multi import BF, U24, close, weight

pytestmark = pytest.mark.gpu


def test_forward(gpu):
    T, K, N, r, n = (1 << 26) - 1, 64, 32, 136, 9
    g = torch.Generator().manual_seed(26)
    rows = torch.tensor([0, 1, 127, 128, (1 << 25) - 1, 1 << 25, T - 129, T - 128, T - 127, T - 2, T - 1])
    S, Wd = weight(N, K, 2, 4, g, gpu)
    A = (torch.randn(n, r, K, generator=g) * 0.05).bfloat16()
    B = (torch.randn(n, N, r, generator=g) * 0.05).bfloat16()
    x = torch.randn(len(rows), K, generator=g).bfloat16()
    ids = torch.randint(-1, n, (T,), generator=g, dtype=torch.int32)
    X = torch.zeros(T, K, dtype=torch.bfloat16, device=gpu)
    X[rows.to(gpu)] = x.to(gpu)
    Y, U = sra.multi_lora_fwd(S, X, A.to(gpu), B.to(gpu), ids.to(gpu))
    i = ids[rows].numpy()
    wy, wu = om.forward(f64(x), Wd, f64(A), f64(B), i)
    sy, su = om.forward(np.abs(f64(x)), np.abs(Wd), np.abs(f64(A)), np.abs(f64(B)), i)
    pick = rows.to(gpu)
    close("U", f64(U[pick]), wu, 40 * U24 * su)
    close("Y", f64(Y[pick]), wy, BF * np.abs(wy) + ((K // 16 + r + 64) * U24 + 2.0 ** -16) * sy)
    for out in (U, Y):  # the others are zero, and written
        assert sum(int(part.any(1).sum()) for part in out.split(1 << 22)) <= len(rows)
