"""Products of 8-bit floating point matrices on the GPU against float64.

Whole numbers whose sums stay below 2^24 (in units of the smallest scale) are exact in fp32 in any order, so most tests
ask for equality.  Others: a sum of K exact products in fp32 is off by at most K U sum |a b| (U = 2^-24) in any order,
and the result by half a step of its type more.
"""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import fp8 as ofp8
from _util import bits, f64

pytestmark = pytest.mark.gpu
KIND = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def whole(R, K, kind, rows, gpu, seed):
    """An operand of small whole numbers (exact in both types) with scales 2^0 .. 2^3."""
    g = torch.Generator().manual_seed(seed)
    blocks = -(-K // 128)
    x = torch.randint(-3, 4, (R, K), generator=g).float()
    codes = torch.zeros(R, blocks * 128)
    codes[:, :K] = x
    exps = torch.randint(127, 131, (-(-R // rows), blocks), generator=g, dtype=torch.uint8)
    F = sra.Fp8Matrix(codes.to(KIND[kind]).to(gpu), exps.to(gpu), R, K, rows)
    s = np.repeat(np.repeat(2.0 ** (exps.numpy().astype(int) - 127), rows, 0)[:R], 128, 1)[:, :K]
    return F, x.numpy().astype(np.float64) * s


def check_whole(M, N, K, ka, kb, ra, rb, gpu, dtype=torch.float32):
    A, a = whole(M, K, ka, ra, gpu, M * 31 + K)
    B, b = whole(N, K, kb, rb, gpu, N * 37 + K + 1)
    got = sra.fp8_matmul(A, B, out_dtype=dtype)
    want = a @ b.T
    assert np.abs(a) .max(initial=0) * np.abs(b).max(initial=0) * K < 2 ** 24
    if dtype == torch.float32:
        assert np.array_equal(f64(got), want)
    else:
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.bfloat16))


SIZES = [(1, 1, 1), (1, 16, 128), (3, 17, 129), (16, 100, 640), (17, 33, 500), (33, 64, 1024), (48, 130, 2000), (64, 257, 384),
         (65, 128, 256), (100, 1000, 4000), (128, 129, 127), (130, 64, 1280), (200, 3, 700), (255, 513, 520), (300, 2100, 900),
         (513, 257, 128), (1025, 300, 1300)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_whole_numbers(gpu, M, N, K):
    check_whole(M, N, K, "e4m3", "e4m3", 1, 128, gpu)
    check_whole(M, N, K, "e5m2", "e4m3", 1, 1, gpu, torch.bfloat16)


@pytest.mark.parametrize("ka", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kb", ["e4m3", "e5m2"])
@pytest.mark.parametrize("ra", [1, 128])
@pytest.mark.parametrize("rb", [1, 128])
def test_kinds_and_blocks(gpu, ka, kb, ra, rb):
    for M, N, K in ((9, 200, 900), (70, 300, 5000), (400, 1500, 600)):
        check_whole(M, N, K, ka, kb, ra, rb, gpu)


def test_large_tiles(gpu):
    """Shapes that fill the GPU with the largest tiles, ragged on both sides."""
    check_whole(4100, 4610, 260, "e4m3", "e4m3", 1, 128, gpu)
    check_whole(4097, 4227, 1281, "e5m2", "e4m3", 1, 1, gpu, torch.bfloat16)


def test_every_code_and_scale(gpu):
    """Each pair of codes of both types once, under scales from one end of the range to the other."""
    for ka in KIND:
        for kb in KIND:
            va, vb = (torch.arange(256, dtype=torch.uint8)[torch.isfinite(torch.from_numpy(ofp8.values(k)))] for k in (ka, kb))
            ca, cb = torch.zeros(len(va), 128, dtype=torch.uint8), torch.zeros(len(vb), 128, dtype=torch.uint8)
            ca[:, 5], cb[:, 5] = va, vb
            for ea, eb in ((1, 127), (127, 127), (246, 20), (60, 190), (239, 4)):
                A = sra.Fp8Matrix(ca.view(KIND[ka]).to(gpu), torch.full((len(va), 1), ea, dtype=torch.uint8, device=gpu), len(va), 128)
                B = sra.Fp8Matrix(cb.view(KIND[kb]).to(gpu), torch.full((len(vb), 1), eb, dtype=torch.uint8, device=gpu), len(vb), 128)
                want = np.outer(ofp8.values(ka)[va.numpy()], ofp8.values(kb)[vb.numpy()]) * 2.0 ** (ea + eb - 254)
                got = f64(sra.fp8_matmul(A, B, out_dtype=torch.float32))
                fine = (np.abs(want) >= 2.0 ** -126) & (np.abs(want) < 2.0 ** 128) | (want == 0)  # not below fp32's normal range
                assert np.array_equal(got[fine], want[fine])


@pytest.mark.parametrize("M,N,K,ka", [(5, 700, 9216, "e4m3"), (64, 300, 3333, "e4m3"), (333, 1024, 4096, "e5m2"), (1000, 640, 2047, "e5m2")])
def test_encoded_operands(gpu, M, N, K, ka):
    g = torch.Generator().manual_seed(M + N + K)
    X, W = torch.randn(M, K, generator=g).to(gpu), torch.randn(N, K, generator=g).to(gpu)
    A, B = sra.fp8_encode(X, KIND[ka]), sra.fp8_encode(W, block_rows=128)
    a, b = f64(sra.fp8_decode(A, torch.float32)), f64(sra.fp8_decode(B, torch.float32))
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    for dtype, half in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)):
        got = f64(sra.fp8_matmul(A, B, out_dtype=dtype))
        assert np.all(np.abs(got - want) <= half * np.abs(want) + K * 2.0 ** -24 * size)
        # and on the whole far nearer: errors of that many roundings add up like a walk, sqrt(K) of them
        assert np.linalg.norm(got - want) <= (half + np.sqrt(K) * 2.0 ** -24) * np.linalg.norm(size)


def test_not_finite_stays_in_its_row(gpu):
    for M, N, K in ((20, 300, 500), (300, 400, 500), (90, 90, 4000)):
        A, a = whole(M, K, "e4m3", 1, gpu, 1)
        B, b = whole(N, K, "e4m3", 1, gpu, 2)
        A.codes.view(torch.uint8)[7, 3] = 0x7F
        B.exps[5, 0] = 255
        got, want = f64(sra.fp8_matmul(A, B, out_dtype=torch.float32)), a @ b.T
        assert np.isnan(got[7]).all() and np.isnan(got[:, 5]).all()
        keep = np.ix_([i for i in range(M) if i != 7], [j for j in range(N) if j != 5])
        assert np.array_equal(got[keep], want[keep])


def test_empty(gpu):
    for M, N, K in ((0, 5, 128), (5, 0, 128), (5, 6, 0), (100, 300, 0), (0, 0, 0)):
        A, _ = whole(M, K, "e4m3", 1, gpu, 1)
        B, _ = whole(N, K, "e4m3", 128, gpu, 2)
        out = torch.full((M, N), 7.0, device=gpu)
        assert not sra.fp8_matmul(A, B, out=out).any()


def test_deterministic_and_given_workspace(gpu):
    A, _ = whole(100, 6000, "e4m3", 1, gpu, 3)
    B, _ = whole(500, 6000, "e4m3", 128, gpu, 4)
    A.codes.view(torch.uint8).random_(0, 0x70)
    want = sra.fp8_matmul(A, B, out_dtype=torch.float32)
    ws = torch.full((sra.fp8_matmul_workspace(100, 500, 6000) + 64,), 0xFF, dtype=torch.uint8, device=gpu)
    for _ in range(3):
        assert np.array_equal(bits(sra.fp8_matmul(A, B, out_dtype=torch.float32, ws=ws)), bits(want))
