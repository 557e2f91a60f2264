"""8-bit products of few rows by few rows over a long reduction: split over the chip, or streamed where that is short.

Whole numbers up to 3 with scales of 1 and 2: sums below 36 K < 2^24, exact in fp32 in any order."""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from _util import f64
from test_gpu_fp8_matmul import KIND

pytestmark = pytest.mark.gpu


def operand(R, K, kind, rows, gpu, seed):
    g = torch.Generator(device=gpu).manual_seed(seed)
    nb = -(-K // 128)
    x = torch.zeros(R, nb * 128, device=gpu)
    x[:, :K] = torch.randint(-3, 4, (R, K), generator=g, device=gpu).float()
    e = torch.randint(127, 129, (-(-R // rows), nb), generator=g, device=gpu, dtype=torch.uint8)
    s = (2.0 ** (e.double() - 127)).repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)
    return sra.Fp8Matrix(x.to(KIND[kind]), e, R, K, rows), x.double() * s


@pytest.mark.parametrize("M,N,K", [(32, 64, 1 << 17), (1, 1, 1 << 17), (16, 256, (1 << 17) - 77), (31, 2048, 16384), (17, 100, 50001),
                                   (7, 33, 16385), (2, 700, 36864), (32, 16, 36863), (32, 70, 300001)])
@pytest.mark.parametrize("ka,rb", [("e4m3", 128), ("e5m2", 1)])
def test_whole_numbers(gpu, M, N, K, ka, rb):
    assert 36 * K < 2 ** 24
    A, a = operand(M, K, ka, 1, gpu, M)
    B, b = operand(N, K, "e4m3", rb, gpu, N)
    want = f64((a @ b.t()).float())
    assert np.array_equal(f64(sra.fp8_matmul(A, B, out_dtype=torch.float32)), want)
    assert torch.equal(sra.fp8_matmul(A, B).cpu(), torch.from_numpy(want).bfloat16())
    A.codes.view(torch.uint8)[M - 1, K - 1] = 0x7F
    got = f64(sra.fp8_matmul(A, B))
    assert np.isnan(got[M - 1]).all() and np.isfinite(got[:M - 1]).all()
