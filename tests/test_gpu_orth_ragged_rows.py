"""Newton-Schulz updates on rows that end inside a vector of loads: what follows a row (the next row, the next matrix, memory
behind the last) is read past neither in sums nor in stores."""
import pytest
import torch

import sparse_rank_adapter_amd as sra

pytestmark = pytest.mark.gpu
SIZES = [(1, 1), (1, 5), (2, 3), (3, 18), (5, 33), (16, 131), (17, 203), (30, 1023), (33, 70), (63, 514), (65, 129), (101, 777),
         (130, 131), (255, 259), (256, 1025)]


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,L", SIZES)
def test_neighbours(gpu, d, L, dt, tall):
    """A matrix between two of NaN, in a buffer of NaN, gives what it gives alone, padded with zeros to whole vectors; and the
    result's neighbours stay as they were."""
    g = torch.Generator().manual_seed(1000 * d + L)
    G = torch.randn(L if tall else d, d if tall else L, generator=g).to(dt)
    R, C = G.shape
    n = R * C
    alone = sra.orthogonalize(G.to(gpu))
    buf = torch.full((3 * n + 64,), float("nan"), dtype=dt)
    buf[n:2 * n] = G.reshape(-1)
    batch = sra.orthogonalize(buf.to(gpu)[:3 * n].view(3, R, C))
    assert torch.equal(batch[1], alone)
    assert torch.isnan(batch[0]).all() and torch.isnan(batch[2]).all()
    out = torch.full((n + 64,), 7.0, dtype=dt, device=gpu)
    sra.orthogonalize(G.to(gpu), out=out[:n].view(R, C))
    assert torch.equal(out[:n].view(R, C), alone) and (out[n:] == 7).all()
    # zero columns along the longer side change no singular value: the same update (another order of fp64 sums, one rounding)
    wide = torch.zeros(R + (16 - R % 16 if tall else 0), C + (0 if tall else 16 - C % 16), dtype=dt)
    wide[:R, :C] = G
    padded = sra.orthogonalize(wide.to(gpu))[:R, :C]
    step = torch.finfo(dt).eps
    assert ((padded.double() - alone.double()).abs() <= step * alone.double().abs() + 1e-9 * alone.double().abs().max()).all()
