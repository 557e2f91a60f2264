"""8-bit codes of rows that end anywhere in a workgroup's four slots of 256 vectors, and of matrices with tiles inside and at
both edges: equal to the oracle's, by each way a matrix is coded."""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import fp8 as ofp8
from _util import f64

pytestmark = pytest.mark.gpu


def raw(F):
    return F.codes.view(torch.uint8).cpu().numpy(), F.exps.cpu().numpy()


def same(F, want):
    return all(np.array_equal(a, b) for a, b in zip(raw(F), want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [8, 120, 1000, 1016, 2040, 2056, 4088, 4104, 6136, 6152, 8184, 8200, 10264, 20488,
                               1, 127, 129, 383, 385, 511, 513, 1025, 1537, 2047, 2049, 2561, 5121])
def test_ends_of_rows(gpu, dtype, C):
    g = torch.Generator().manual_seed(C)
    X = (torch.randn(3, C, generator=g) * torch.exp(2 * torch.randn(3, C, generator=g))).to(dtype)
    want = ofp8.encode(f64(X), "e4m3", 1)
    assert same(sra.fp8_encode(X.to(gpu)), want)
    F, Ft = sra.fp8_encode_pair(X.to(gpu))
    assert same(F, want)
    if C < 1000:
        assert same(Ft, ofp8.encode(f64(X).T, "e4m3", 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", [(256, 256), (300, 264), (255, 256), (256, 255), (129, 392), (128, 128), (270, 129)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_tiles_inside_and_at_the_edges(gpu, dtype, R, C, block_rows):
    g = torch.Generator().manual_seed(R + C)
    X = (torch.randn(R, C, generator=g) * torch.exp(2 * torch.randn(R, 1, generator=g))).to(dtype)
    X[R - 1, C - 1], X[0, 0] = float("inf"), float("nan")
    F, Ft = sra.fp8_encode_pair(X.to(gpu), torch.float8_e5m2, block_rows=block_rows)
    codes, exps = ofp8.encode(f64(X), "e5m2", block_rows)
    for f, c, e in ((F, codes, exps), (Ft, *ofp8.encode(f64(X).T, "e5m2", block_rows))):
        got, ge = raw(f)
        assert np.array_equal(ge, e)
        nan = np.isnan(ofp8.values("e5m2")[c])
        assert np.array_equal(got[~nan], c[~nan]) and np.isnan(ofp8.values("e5m2")[got[nan]]).all()
