"""8-bit floating point matrices on the GPU: codes and scales equal the float64 oracle's, bit for bit."""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import fp8 as ofp8
from _util import f64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
KIND = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def data(R, C, dtype, gpu):
    g = torch.Generator().manual_seed(R * 1009 + C)
    size = torch.exp2(torch.randint(-30, 30, (R, 1), generator=g).float()) * torch.exp2(torch.randint(-6, 6, (1, C), generator=g).float())
    return (torch.randn(R, C, generator=g) * size).to(DT[dtype]).to(gpu)


def raw(F):
    return F.codes.view(torch.uint8).cpu().numpy(), F.exps.cpu().numpy()


def check(F, X64, kind, block_rows):
    codes, exps = ofp8.encode(X64, kind, block_rows)
    assert np.array_equal(F.exps.cpu().numpy(), exps)
    assert np.array_equal(F.codes.view(torch.uint8).cpu().numpy(), codes)
    want = ofp8.decode(codes, exps, kind, X64.shape[1], block_rows)
    assert np.array_equal(f64(sra.fp8_decode(F, torch.float32)), want, equal_nan=True)
    assert np.array_equal(f64(sra.fp8_decode(F)), want, equal_nan=True)  # 4 bits or fewer: exact in bf16


SHAPES = [(1, 1), (1, 127), (2, 128), (3, 129), (7, 256), (128, 128), (127, 130), (129, 264), (130, 1001), (257, 384),
          (1, 5000), (300, 8), (1000, 33)]


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", SHAPES)
def test_encode_decode(gpu, R, C, dtype, kind):
    X = data(R, C, dtype, gpu)
    x = f64(X)
    for rows in (1, 128):
        check(sra.fp8_encode(X, KIND[kind], rows), x, kind, rows)
        F, Ft = sra.fp8_encode_pair(X, KIND[kind], rows)
        check(F, x, kind, rows)
        check(Ft, x.T, kind, rows)
        T = sra.fp8_encode_t(X, KIND[kind], rows)
        for a, b in zip(raw(T), raw(Ft)):
            assert np.array_equal(a, b)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows", [1, 128])
def test_every_rounding_and_border(gpu, kind, rows):
    """Every value of the type, the midpoints between neighbours and the fp32 values next to them, in blocks whose
    largest value is at, just under and just over the border to the next scale."""
    v = ofp8.values(kind)[:ofp8.KINDS[kind][3] + 1]
    mid = ((v[1:] + v[:-1]) / 2).astype(np.float32)
    line = np.concatenate([v.astype(np.float32), mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e30))])
    lim = np.float32(v[-1])
    tops = [lim, np.nextafter(lim, np.float32(0)), np.nextafter(lim, np.float32(1e30)), lim / 2, np.nextafter(lim / 2, np.float32(1e30))]
    out = []
    for t in tops:
        for e in (-100, -3, 0, 60):
            for i in range(0, line.size, 127):
                row = np.zeros(128, np.float32)
                part = line[i:i + 127]
                row[:part.size] = np.where(part <= t, part, 0) * np.where(np.arange(part.size) % 3 == 0, -1, 1)
                row[127] = t
                out.append(np.ldexp(row, e).astype(np.float32))
    X = torch.from_numpy(np.stack(out)).to(gpu)
    check(sra.fp8_encode(X, KIND[kind], rows), f64(X), kind, rows)
    F, Ft = sra.fp8_encode_pair(X, KIND[kind], rows)
    check(Ft, f64(X).T, kind, rows)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows", [1, 128])
def test_not_finite_extreme_and_signed_zero(gpu, kind, rows):
    X = data(260, 300, "f32", gpu)
    X[0, 3], X[1, 200], X[2, 10] = float("nan"), float("inf"), -float("inf")
    X[3] = float("inf")
    X[4] = 3.4e38  # past the largest scale: saturates
    X[5] = 1e-42   # below the smallest scale's smallest value
    X[6] = -0.0
    X[7, 0], X[7, 1] = 2.0 ** -126, -2.0 ** -127
    x = f64(X)
    F, Ft = sra.fp8_encode_pair(X, KIND[kind], rows)
    for f, want in ((F, x), (Ft, x.T), (sra.fp8_encode(X, KIND[kind], rows), x)):
        codes, exps = ofp8.encode(want, kind, rows)
        got, e = raw(f)
        assert np.array_equal(e, exps)
        live = np.zeros(codes.shape, bool)
        live[:, :want.shape[1]] = ~np.isfinite(want)
        assert np.array_equal(got[~live], codes[~live])
        assert np.isnan(ofp8.values(kind)[got[live]]).all()  # any of the type's NaN codes


def test_scales_past_the_encoders_range(gpu):
    """Exponent bytes that the encoder never writes keep their E8M0 meaning: 0 is 2^-127, 255 is NaN."""
    codes = torch.full((3, 128), 0x38, dtype=torch.uint8, device=gpu)  # 1.0
    F = sra.Fp8Matrix(codes.view(torch.float8_e4m3fn), torch.tensor([[0], [254], [255]], dtype=torch.uint8, device=gpu), 3, 128)
    x = sra.fp8_decode(F, torch.float32)
    assert (x[0] == 2.0 ** -127).all() and (x[1] == 2.0 ** 127).all() and torch.isnan(x[2]).all()


def test_into_given_buffers_and_empty(gpu):
    X = data(50, 200, "bf16", gpu)
    F, Ft = sra.fp8_encode_pair(X)
    want = [raw(F), raw(Ft)]
    for t in (F.codes.view(torch.uint8), F.exps, Ft.codes.view(torch.uint8), Ft.exps):
        t.fill_(0x55)
    sra.fp8_encode_pair(X, out=(F, Ft))
    for f, w in zip((F, Ft), want):
        assert all(np.array_equal(a, b) for a, b in zip(raw(f), w))
    for R, C in ((0, 5), (5, 0)):
        Z = torch.zeros(R, C, device=gpu)
        F, Ft = sra.fp8_encode_pair(Z)
        assert F.shape == (R, C) and Ft.shape == (C, R) and sra.fp8_decode(F).shape == (R, C)


def test_more_than_2_31_codes(gpu):
    """Offsets past 32 bits, in rows and in the transpose."""
    R, C = 40000, 65536
    X = torch.zeros(R, C, dtype=torch.bfloat16, device=gpu)
    X[-1, -130:] = 3.0
    X[-129, 7] = -5.0
    F, Ft = sra.fp8_encode_pair(X)
    codes, exps = ofp8.encode(f64(X[-200:]), "e4m3")
    assert np.array_equal(F.codes[-200:].view(torch.uint8).cpu().numpy(), codes) and np.array_equal(F.exps[-200:].cpu().numpy(), exps)
    tail = f64(X[-256 - R % 128:, -130:].t())  # whole blocks of the transpose's rows
    codes, exps = ofp8.encode(tail, "e4m3")
    n = codes.shape[1]
    assert np.array_equal(Ft.codes[-130:, -n:].view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(Ft.exps[-130:, -n // 128:].cpu().numpy(), exps)
    del Ft
    back = sra.fp8_decode(F, out=X)
    assert torch.equal(back[-1, -130:], torch.full((130,), 3.0, dtype=X.dtype, device=gpu)) and back[-129, 7] == -5.0
    assert not back[:-129].any()
