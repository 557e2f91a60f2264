"""Layer norm over more rows than one launch of a workgroup per row can take: 2^26 rows of 64 threads are 2^32
threads.  A row's results depend on the row alone, so rows at both ends and around the launches' borders are
compared with a call on those rows only; the backward's sums are compared with the float64 ones."""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from _util import f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("T,H,ckpt", [((1 << 26) + 5, 8, True), ((1 << 22) + 3, 2056, False), ((1 << 21) + 1, 33, True)])
def test_rows(gpu, T, H, ckpt):
    g = torch.Generator().manual_seed(H)
    border = 1 << 21
    rows = sorted({t for t in (0, 1, border - 1, border, border + 1, 2 * border - 1, 2 * border, 2 * border + 2,
                               16 * border, 31 * border + 7, T - 2, T - 1) if t < T})
    pick = torch.tensor(rows, device=gpu)
    x = torch.randn(len(rows), H, generator=g).bfloat16().to(gpu)
    dy = torch.randn(len(rows), H, generator=g).bfloat16().to(gpu)
    gamma, beta = (torch.randn(H, generator=g).bfloat16().to(gpu) for _ in range(2))
    X = torch.ones(T, H, dtype=torch.bfloat16, device=gpu)
    X[pick] = x
    Y, mean, rstd, c = sra.layer_norm_fwd(X, gamma, beta, ckpt=ckpt)
    y1, m1, r1, c1 = sra.layer_norm_fwd(x, gamma, beta, ckpt=ckpt)
    assert torch.equal(Y[pick], y1) and torch.equal(mean[pick], m1) and torch.equal(rstd[pick], r1)
    if ckpt:
        assert torch.equal(c.codes[pick], c1.codes) and torch.equal(c.exps[pick], c1.exps)
    # every other row is of ones: mean 1, no deviation
    assert int((mean != 1).sum()) <= len(rows)
    assert sum(int((part != beta).any(1).sum()) for part in Y.split(1 << 19)) <= len(rows)
    del Y, c

    dY = torch.zeros(T, H, dtype=torch.bfloat16, device=gpu)
    dY[pick] = dy
    dX, dg, db = sra.layer_norm_bwd(dY, X, gamma, mean, rstd)
    assert torch.equal(dX[pick], sra.layer_norm_bwd(dy, x, gamma, m1, r1)[0])
    # fp32 sums of len(rows) terms that are not zero, three roundings a term
    d, xh = f64(dy), (f64(x) - f64(m1)[:, None]) * f64(r1)[:, None]
    size = np.abs(xh) + np.abs(f64(m1) * f64(r1))[:, None]
    assert np.all(np.abs(f64(dg) - (d * xh).sum(0)) <= (len(rows) + 4) * U * np.abs(d * size).sum(0))
    assert np.all(np.abs(f64(db) - d.sum(0)) <= (len(rows) + 1) * U * np.abs(d).sum(0))
