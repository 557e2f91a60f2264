"""The many-adapter decode kernels (16 tokens or fewer): every workgroup shape, both layouts, 2:4 and 2:8 weights.

Tolerances as in test_gpu_multi."""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import multi as om
from _util import bits, f64
from test_gpu_multi import BF, U24, close, make_ids, weight

pytestmark = pytest.mark.gpu


def check(gpu, T, R, C, r, n, fmt, tiled, kind, rows=0):
    g = torch.Generator().manual_seed(T + R + C + r)
    S, D = weight(R, C, *fmt, g, gpu)
    if tiled:
        S = sra.nm_tile(S)
    X = torch.randn(T, C, generator=g).bfloat16().to(gpu)
    A = (torch.randn(n, r, C, generator=g) * 0.05).bfloat16().to(gpu)
    B = (torch.randn(n, R, r, generator=g) * 0.05).bfloat16().to(gpu)
    ids = make_ids(kind, T, n, g)
    di = ids.to(gpu)
    with sra.tuned(decode_rows=rows):
        Y, U = sra.multi_lora_fwd(S, X, A, B, di)
        order = torch.argsort(di, stable=True)
        Y2, U2 = sra.multi_lora_fwd(S, X[order].contiguous(), A, B, di[order].contiguous())
    x, a, b = f64(X), f64(A), f64(B)
    wy, wu = om.forward(x, D, a, b, ids.numpy())
    sy, su = om.forward(np.abs(x), np.abs(D), np.abs(a), np.abs(b), ids.numpy())
    close("U", f64(U), wu, 40 * U24 * su)
    close("Y", f64(Y), wy, BF * np.abs(wy) + ((C // 16 + r + 64) * U24 + 2.0 ** -16) * sy)
    assert np.array_equal(bits(Y2), bits(Y[order])) and np.array_equal(bits(U2), bits(U[order]))


@pytest.mark.parametrize("fmt", [(2, 4), (2, 8)])
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("rows", [3, 4, 9])
@pytest.mark.parametrize("T,R,C,r,kind", [(1, 300, 160, 8, "one"), (7, 330, 608, 40, "mixed"), (16, 1000, 544, 10, "mixed"),
                                          (16, 145, 1024, 130, "requests")])
def test_shapes(gpu, T, R, C, r, kind, rows, tiled, fmt):
    check(gpu, T, R, C, r, 1 if kind == "one" else 12, fmt, tiled, kind, rows)


@pytest.mark.parametrize("fmt", [(2, 4), (2, 8)])
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("R", [4000, 12300, 16400, 36864])
def test_own_choice(gpu, R, tiled, fmt):
    check(gpu, 16, R, 128, 24, 9, fmt, tiled, "mixed")
