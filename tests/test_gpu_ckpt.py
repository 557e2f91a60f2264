"""8-bit activation checkpoints on the GPU against the oracle: codes, exponents and values bit for bit."""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import ckpt as ock
from _util import f64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def check(X):
    c = sra.ckpt8_encode(X)
    codes, exps = ock.encode(f64(X))
    assert np.array_equal(c.exps.cpu().numpy(), exps)
    assert np.array_equal(c.codes.cpu().numpy(), codes)
    V = sra.ckpt8_decode(c)
    assert V.dtype == X.dtype
    assert np.array_equal(f64(V), ock.decode(codes, exps))  # exact in either type


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K", [(1, 1), (1, 31), (1, 32), (3, 33), (2, 40), (5, 64), (7, 95), (4, 130), (33, 1024),
                                 (2, 8193), (3, 4098), (1, 20480), (40000, 8), (17, 2056)])
def test_roundtrip(gpu, dtype, T, K):
    g = torch.Generator().manual_seed(T * 131 + K)
    X = torch.randn(T, K, generator=g) * torch.where(torch.rand(K, generator=g) < 0.05, 30.0, 1.0)
    check(X.to(DT[dtype]).to(gpu))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_edges(gpu, dtype):
    """Zero blocks, the scale's borders (127 2^k and the next value up), halves, subnormals, the largest values."""
    big = float(torch.finfo(DT[dtype]).max)
    tiny = float(torch.finfo(DT[dtype]).smallest_normal)
    X = torch.zeros(12, 96)
    X[1, 5] = 127.0
    X[2, 5] = 127.5 if dtype == "bf16" else float(np.nextafter(np.float32(127), np.float32(128)))
    X[3, :32] = torch.arange(32) + 0.5        # ties: 0.5 -> 0, 1.5 -> 2, ...
    X[3, 31] = 127.0
    X[4, 0], X[4, 1], X[4, 40] = big, -big, 1.0
    X[5, :3] = torch.tensor([tiny, -tiny, tiny / 2])
    X[6, 0] = tiny / 64
    X[7, 33] = -0.0
    X[8] = torch.linspace(-3, 3, 96)
    X[9, 95] = -254.0
    X[10, 64:] = 2.0 ** -100
    X[11, 0] = 127 * 2.0 ** -126
    check(X.to(DT[dtype]).to(gpu))


def test_empty(gpu):
    for T, K in ((0, 64), (4, 0)):
        c = sra.ckpt8_encode(torch.zeros(T, K, dtype=torch.bfloat16, device=gpu))
        assert sra.ckpt8_decode(c).shape == (T, K)


def test_other_stream(gpu):
    X = torch.randn(64, 256, device=gpu).bfloat16()
    want = sra.ckpt8_decode(sra.ckpt8_encode(X))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = sra.ckpt8_decode(sra.ckpt8_encode(X))
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
