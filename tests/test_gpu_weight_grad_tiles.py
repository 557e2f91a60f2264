"""The masked weight gradient on its 128-row workgroups (from 256 of them) with ragged edges, from bf16 and from a
checkpoint, against float64.  Tolerance: half a bf16 step of the result, and fp32 sums of 64 tokens between
the fp64 additions (64 + 6 roundings of 2^-24 of the sum of magnitudes)."""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from _util import bits, f64

pytestmark = pytest.mark.gpu
U24, BF = 2.0 ** -24, 2.0 ** -8


@pytest.mark.parametrize("T", [1, 63, 70, 200])
@pytest.mark.parametrize("R,C", [(4104, 1056), (4096, 1024), (8, 32768), (32760, 96)])
def test_ragged(gpu, T, R, C):
    g = torch.Generator().manual_seed(T + R)
    S = sra.compress((torch.randn(R, C, generator=g) * 0.05).bfloat16().to(gpu))
    dY = torch.randn(T, R, generator=g).bfloat16().to(gpu)
    X = torch.randn(T, C, generator=g).bfloat16().to(gpu)
    kept = sra.ckpt8_encode(X)
    words = S.meta.cpu().numpy().view(np.uint32)
    i = np.arange(C // 2)
    col = (i // 2) * 4 + ((words[:, i // 16] >> (2 * (i % 16)).astype(np.uint32)) & 3)
    from_kept = None
    for act in (X, sra.ckpt8_decode(kept)):
        got = sra.masked_weight_grad(S, dY, act)
        w = np.take_along_axis(f64(dY).T @ f64(act), col, 1)
        mag = np.take_along_axis(np.abs(f64(dY)).T @ np.abs(f64(act)), col, 1)
        assert np.all(np.abs(f64(got) - w) <= BF * np.abs(w) + 70 * U24 * mag)
        from_kept = got
    assert np.array_equal(bits(sra.masked_weight_grad(S, dY, kept)), bits(from_kept))
