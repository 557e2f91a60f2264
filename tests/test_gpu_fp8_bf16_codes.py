"""Products of 8-bit floating point matrices with bf16 results: every code, every end of the scales' range, NaN codes and
scales, in each kernel.  (fp32 results widen the codes to bf16 and apply the scales themselves; bf16 results leave both to the
matrix instruction.)

A product of two codes has at most 8 significant bits, so alone in its sum it is exact in bf16."""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import fp8 as ofp8
from _util import f64
from test_gpu_fp8_matmul import KIND, whole

pytestmark = pytest.mark.gpu
# rows of a per call, knob: the streaming kernel with one fragment of a and with two, then each tile
KERNELS = [(16, 0), (32, 0), (None, 64), (None, 128), (None, 132), (None, 256)]


def product(A, B, rows, tile):
    """a b^T in bf16, `rows` rows of a at a time (None: all at once)."""
    step = rows or A.rows
    out = []
    for lo in range(0, A.rows, step):
        part = sra.Fp8Matrix(A.codes[lo:lo + step].clone(), A.exps[lo:lo + step].clone(), min(step, A.rows - lo), A.cols)
        with sra.tuned(fp8_tile=tile):
            out.append(sra.fp8_matmul(part, B))
    return torch.cat(out)


@pytest.mark.parametrize("rows,tile", KERNELS)
@pytest.mark.parametrize("ka", KIND)
@pytest.mark.parametrize("kb", KIND)
def test_every_code_and_scale(gpu, rows, tile, ka, kb):
    va, vb = (torch.arange(256, dtype=torch.uint8)[torch.isfinite(torch.from_numpy(ofp8.values(k)))] for k in (ka, kb))
    ca, cb = torch.zeros(len(va), 256, dtype=torch.uint8), torch.zeros(len(vb), 256, dtype=torch.uint8)
    ca[:, 133], cb[:, 133] = va, vb  # in the second of two blocks, whose scales vary
    most = float(torch.finfo(torch.bfloat16).max)
    for ea, eb in ((1, 127), (127, 127), (246, 20), (60, 190), (239, 4), (254, 0), (0, 254), (0, 200), (200, 1), (254, 100), (130, 120)):
        E = lambda n, e: torch.tensor([[127, e]], dtype=torch.uint8, device=gpu).repeat(n, 1)
        A = sra.Fp8Matrix(ca.view(KIND[ka]).to(gpu), E(len(va), ea), len(va), 256)
        B = sra.Fp8Matrix(cb.view(KIND[kb]).to(gpu), E(len(vb), eb), len(vb), 256)
        want = np.outer(ofp8.values(ka)[va.numpy()], ofp8.values(kb)[vb.numpy()]) * 2.0 ** (ea + eb - 254)
        got = f64(product(A, B, rows, tile))
        fine = (np.abs(want) >= 2.0 ** -126) & (np.abs(want) <= most) | (want == 0)  # inside bf16's normal range
        assert np.array_equal(got[fine], want[fine]), (ea, eb)


@pytest.mark.parametrize("rows,tile", KERNELS)
@pytest.mark.parametrize("K", [256, 500, 4000])
def test_not_finite_stays_in_its_row(gpu, rows, tile, K):
    M, N = rows or 300, 400
    bad_a, bad_b = {7: "code", M - 1: "scale"}, {5: "scale", 130: "code", N - 1: "code"}
    A, a = whole(M, K, "e5m2", 1, gpu, K)
    B, b = whole(N, K, "e4m3", 1, gpu, K + 1)
    for F, bad, col in ((A, bad_a, 3), (B, bad_b, K - 1)):
        for r, what in bad.items():
            if what == "code":
                F.codes.view(torch.uint8)[r, col] = 0x7F
            else:
                F.exps[r, col // 128] = 255
    got, want = product(A, B, rows, tile).cpu(), torch.from_numpy(a @ b.T).bfloat16()
    keep_a, keep_b = [i for i in range(M) if i not in bad_a], [j for j in range(N) if j not in bad_b]
    assert torch.isnan(got[list(bad_a)]).all() and torch.isnan(got[:, list(bad_b)]).all()
    assert torch.equal(got[keep_a][:, keep_b], want[keep_a][:, keep_b])


def test_not_finite_stays_in_its_tile(gpu):
    """256 x 256 tiles, more of them than workgroups: what an earlier tile of a workgroup held does not reach its next."""
    M, N, K = 256 * 9 + 40, 256 * 32 + 24, 300
    A, a = whole(M, K, "e4m3", 1, gpu, 5)
    B, b = whole(N, K, "e4m3", 1, gpu, 6)
    bad_a, bad_b = [3, 700, 2000], [5, 255, 4000, N - 1]
    A.codes.view(torch.uint8)[bad_a, 290] = 0x7F
    B.exps[bad_b, 0] = 255
    with sra.tuned(fp8_tile=256):
        got = sra.fp8_matmul(A, B)
    want = (torch.from_numpy(a).to(gpu) @ torch.from_numpy(b).to(gpu).t()).bfloat16()
    assert torch.isnan(got[bad_a]).all() and torch.isnan(got[:, bad_b]).all()
    want[bad_a], want[:, bad_b] = 0.0, 0.0
    got[bad_a], got[:, bad_b] = 0.0, 0.0
    assert torch.equal(got, want)


def test_infinities(gpu):
    """e5m2's infinity, which the encoder does not write: its row's results are infinite or NaN, the others as ever."""
    A, a = whole(300, 384, "e5m2", 1, gpu, 7)
    B, b = whole(400, 384, "e4m3", 1, gpu, 8)
    A.codes.view(torch.uint8)[9, 200] = 0x7C
    want = torch.from_numpy(a @ b.T).bfloat16()
    for rows, tile in KERNELS:
        got = product(A, B, rows, tile).cpu()
        assert not torch.isfinite(got[9]).any()
        rest = [i for i in range(300) if i != 9]
        assert torch.equal(got[rest], want[rest])
