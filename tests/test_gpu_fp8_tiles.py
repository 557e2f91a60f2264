"""Every tile of the 8-bit floating point product, over ragged shapes, kinds and both result types: whole numbers whose
sums are exact, so every tile gives the same."""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from _util import bits, f64
from test_gpu_fp8_matmul import KIND, whole

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tile", [64, 128, 132, 256])
@pytest.mark.parametrize("ka,kb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_tile(gpu, tile, ka, kb):
    for M, N, K, ra, rb in ((1, 1, 1, 1, 128), (33, 70, 130, 1, 1), (256, 256, 512, 128, 128), (257, 300, 1000, 1, 128), (300, 264, 640, 1, 1),
                            (129, 515, 2100, 128, 1), (700, 40, 385, 1, 128), (64, 1000, 2200, 1, 1)):
        A, a = whole(M, K, ka, ra, gpu, M + K)
        B, b = whole(N, K, kb, rb, gpu, N + K + 1)
        with sra.tuned(fp8_tile=tile):
            f = sra.fp8_matmul(A, B, out_dtype=torch.float32)
            h = sra.fp8_matmul(A, B)
        want = a @ b.T
        assert np.array_equal(f64(f), want), (M, N, K)
        assert torch.equal(h.cpu(), torch.from_numpy(want).to(torch.bfloat16)), (M, N, K)


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 15, 16, 17, 18, 20, 31, 33])
def test_lengths_of_the_reduction_with_several_tiles_a_workgroup(gpu, blocks):
    """256 x 256 tiles, more of them than workgroups: rings and scales run on from tile to tile."""
    M, N, K = 256 * 9 + 40, 256 * 32 + 24, 128 * blocks - (37 if blocks % 2 else 0)
    A, a = whole(M, K, "e4m3", 1, gpu, blocks)
    B, b = whole(N, K, "e4m3", 128, gpu, blocks + 1)
    with sra.tuned(fp8_tile=256):
        got = sra.fp8_matmul(A, B)
    a, b = torch.from_numpy(a).to(gpu), torch.from_numpy(b).to(gpu)
    assert torch.equal(got, (a @ b.t()).to(torch.bfloat16))


@pytest.mark.parametrize("tile", [64, 128, 132, 256])
def test_rows_behind_the_matrix_are_left_alone(gpu, tile):
    A, _ = whole(300, 700, "e4m3", 1, gpu, 1)
    for N in (264, 260, 257):  # stores of 8 columns, of 4, of one
        B, _ = whole(N, 700, "e4m3", 128, gpu, 2)
        for dtype in (torch.bfloat16, torch.float32):
            buf = torch.full((310 * N,), 7.0, dtype=dtype, device=gpu)
            out = buf[:300 * N].view(300, N)
            with sra.tuned(fp8_tile=tile):
                sra.fp8_matmul(A, B, out=out)
            assert (buf[300 * N:] == 7.0).all()
            assert torch.equal(out, sra.fp8_matmul(A, B, out_dtype=dtype))


def test_fp32_results_keep_small_products_beside_large_ones(gpu):
    """2^23 and up to 127 ones in a block: exact in fp32, lost where products are aligned to the largest with 17 bits."""
    for M, N, nb in ((20, 50, 1), (200, 300, 3), (20, 50, 9)):
        a, b = torch.zeros(M, 128 * nb), torch.zeros(N, 128 * nb)
        a[:, 64], b[:, 64] = 32768.0, 256.0
        for i in range(127):
            k = i if i < 64 else i + 1
            a[i % M:, k], b[:, k] = 1.0, 1.0
        E = lambda n: torch.full((n, nb), 127, dtype=torch.uint8, device=gpu)
        A = sra.Fp8Matrix(a.to(torch.float8_e5m2).to(gpu), E(M), M, 128 * nb)
        B = sra.Fp8Matrix(b.to(torch.float8_e4m3fn).to(gpu), E(N), N, 128 * nb)
        want = a.double().numpy() @ b.double().numpy().T
        assert want.max() < 2 ** 24
        assert np.array_equal(f64(sra.fp8_matmul(A, B, out_dtype=torch.float32)), want)
        for tile in (64, 128):
            with sra.tuned(fp8_tile=tile):
                assert np.array_equal(f64(sra.fp8_matmul(A, B, out_dtype=torch.float32)), want)


def test_scales_at_the_end_of_their_array(gpu):
    """Rows of 1 to 5 blocks: the last rows' scales are read up to the array's last byte, which lies before other data."""
    for nb in (1, 2, 3, 5):
        for M in (1, 2, 3, 40, 129):
            store = torch.full((M * nb + 64,), 255, dtype=torch.uint8, device=gpu)  # 255 would give NaN
            A, a = whole(M, 128 * nb, "e4m3", 1, gpu, M + nb)
            store[:M * nb] = A.exps.flatten()
            A.exps = store[:M * nb].view(M, nb)
            B, b = whole(70, 128 * nb, "e4m3", 128, gpu, nb)
            for tile in (0, 64, 128, 132, 256):
                with sra.tuned(fp8_tile=tile):
                    assert np.array_equal(f64(sra.fp8_matmul(A, B, out_dtype=torch.float32)), a @ b.T)
                    assert torch.equal(sra.fp8_matmul(A, B).cpu(), torch.from_numpy(a @ b.T).to(torch.bfloat16))
