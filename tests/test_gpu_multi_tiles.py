"""Every tile of the many-adapter product, in both layouts: the forward's Y and the backward's dX against float64.

The plan takes 256 x 256 tiles from 512 of them, 256 x 128 from 129 of those, and small ones below; reductions of
whole 128 columns read their metadata in super-stages, odd multiples of 64 by the stage, odd multiples of 32 take
the register-staged tile.  Tolerances as in test_gpu_multi.
"""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from _util import bits, f64
from test_gpu_multi import BF, U24, close, make_ids, weight

pytestmark = pytest.mark.gpu

# tokens, rows, reduction, rank, adapters, streaming layout
HUGE = [(4100, 8192, 128, 40, 5, True), (4100, 8192, 384, 136, 3, True), (4100, 8192, 640, 10, 40, True),
        (4100, 8192, 128, 136, 3, False), (4100, 8160, 256, 40, 7, False), (4100, 8192, 640, 10, 40, False),
        (4100, 8192, 192, 40, 5, False), (4100, 8192, 64, 136, 3, False), (33000, 1024, 256, 16, 6, True)]
MIDDLE = [(1300, 4096, 128, 40, 5, True), (1300, 4096, 640, 136, 12, True), (1300, 4096, 640, 10, 40, False),
          (1300, 4096, 192, 40, 5, False), (1300, 4000, 64, 136, 12, False)]
SMALL = [(700, 2048, 256, 40, 5, True), (700, 2048, 256, 136, 20, False), (300, 384, 192, 10, 5, False),
         (100, 200, 1088, 40, 9, False), (1000, 2048, 96, 24, 5, False)]


def product(act, W, E, V, ids):
    """act W^T plus every adapter's V_g E_g^T, V_g [T', r] given for all tokens as V [T, r]"""
    out = act @ W.T
    for g in range(E.shape[0]):
        t = ids == g
        out[t] += V[t] @ E[g].T
    return out


@pytest.mark.parametrize("kind", ["mixed", "requests"])
@pytest.mark.parametrize("T,R,C,r,n,tiled", HUGE + MIDDLE + SMALL)
def test_products(gpu, T, R, C, r, n, tiled, kind):
    g = torch.Generator().manual_seed(T + R + C + r)
    S, D = weight(R, C, 2, 4, g, gpu)
    if tiled:
        S = sra.nm_tile(S)
    act = torch.randn(T, C, generator=g).bfloat16().to(gpu)
    wide = (torch.randn(n, r, R, generator=g) * 0.05).bfloat16()  # A of the backward, B^T of the forward
    narrow = (torch.randn(n, r, C, generator=g) * 0.05).bfloat16()
    ids = make_ids(kind, T, n, g)
    di, i, x, w = ids.to(gpu), ids.numpy(), f64(act), f64(wide).transpose(0, 2, 1)
    steps = C // 16 + r + 64

    A, B = narrow.to(gpu), wide.transpose(1, 2).contiguous().to(gpu)
    Y, U = sra.multi_lora_fwd(S, act, A, B, di)
    mag = product(np.abs(x), np.abs(D), np.abs(w), np.abs(f64(U)), i)
    want = product(x, D, w, f64(U), i)  # of the U that the product read
    close("Y", f64(Y), want, BF * np.abs(want) + (steps * U24 + 2.0 ** -16) * mag)

    A, B = wide.to(gpu), narrow.transpose(1, 2).contiguous().to(gpu)
    got = sra.multi_lora_bwd(S, act, None, None, A, B, di, da=False, db=False, want_du=True)
    mag = product(np.abs(x), np.abs(D), np.abs(w), np.abs(f64(got["dU"])), i)
    want = product(x, D, w, f64(got["dU"]), i)
    close("dX", f64(got["dX"]), want, BF * np.abs(want) + (steps * U24 + 2.0 ** -16) * mag)

    # a token's bits do not depend on its neighbours: in another order, and beside an adapter of infinities
    order = torch.argsort(di, stable=True)
    again = sra.multi_lora_bwd(S, act[order].contiguous(), None, None, A, B, di[order].contiguous(), da=False, db=False,
                               want_du=True)
    for k in ("dU", "dX"):
        assert np.array_equal(bits(again[k]), bits(got[k][order].contiguous())), k
    A2, others = A.clone(), di != 1
    A2[1] = float("inf")
    loud = sra.multi_lora_bwd(S, act, None, None, A2, B, di, da=False, db=False)["dX"]
    assert np.array_equal(bits(loud[others].contiguous()), bits(got["dX"][others].contiguous()))
