"""Root-mean-square norm on the GPU against the float64 oracle.

Tolerances count roundings of half a unit in the last place (U = 2^-24, relative): h = x + r one; a thread's sum of up
to 16 squares one for the square and four for the tree, two for h's own; rstd one more and half of the sum's: 6 U.  y =
h rstd gamma: 1 + 6 + 2 = 9 U, and half a step of the output's type (bf16 2^-8, fp32 2^-24).  The backward's sum is of up
to 16 fused steps a thread on terms with three roundings each: 19 U.
"""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import fp8 as ofp8
from oracle import rms as orms
from _util import bits, f64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24
EPS = 1e-6


def data(T, H, dtype, gpu):
    g = torch.Generator().manual_seed(T * 977 + H)
    t = lambda *s, sd=1.0, m=0.0: (torch.randn(*s, generator=g) * sd + m).to(DT[dtype]).to(gpu)
    return t(T, H), t(T, H, sd=0.5), t(H, sd=0.1, m=1.0), t(T, H), t(T, H)


def check_fwd(X, R, gamma, dtype, fp8=True, want_y=True):
    Y, Hs, rstd, F = sra.rms_norm_fwd(X, gamma, EPS, residual=R, fp8=torch.float8_e4m3fn if fp8 else None, want_y=want_y)
    y, h, rs = orms.forward(f64(X), None if R is None else f64(R), f64(gamma), EPS)
    if R is None:
        assert Hs is X
    else:
        assert np.all(np.abs(f64(Hs) - h) <= (HALF[dtype] + U * (1 + HALF[dtype])) * np.abs(h))
    assert np.all(np.abs(f64(rstd) - rs) <= 6 * U * rs)
    if want_y:
        assert np.all(np.abs(f64(Y) - y) <= (HALF[dtype] + 9 * U * (1 + HALF[dtype])) * np.abs(y))
    else:
        assert Y is None
    if fp8:
        W = X.shape[1]
        codes, exps = F.codes.view(torch.uint8).cpu().numpy(), F.exps.cpu().numpy()
        assert not codes[:, W:].any()
        scale = 2.0 ** (exps.astype(np.int64) - 127)
        top = np.stack([np.abs(y[:, b:b + 128]).max(1) for b in range(0, W, 128)], 1)
        assert np.all(top <= 448 * scale * (1 + 9 * U))
        assert np.all((top > 224 * scale * (1 - 9 * U)) | (exps == 1))
        step = np.repeat(scale, 128, axis=1)[:, :W]
        err = np.abs(ofp8.decode(codes, exps, "e4m3", W) - y)
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * step) + 10 * U * np.abs(y) + 10 * U * step)
        if want_y and dtype == "f32":  # the codes are those of the fp32 values
            want = ofp8.encode(f64(Y), "e4m3")
            assert np.array_equal(codes, want[0]) and np.array_equal(exps, want[1])
    else:
        assert F is None
    return Hs, rstd


def check_bwd(dY, Hs, gamma, rstd, dH, dtype):
    dX, dg = sra.rms_norm_bwd(dY, Hs, gamma, rstd, dH=dH)
    dy, h, ga, rs = f64(dY), f64(Hs), f64(gamma), f64(rstd)
    wx, wg = orms.backward(dy, h, ga, rs, None if dH is None else f64(dH))
    xh, g = np.abs(h * rs[:, None]), np.abs(dy * ga)
    terms = rs[:, None] * (g + xh * (g * xh).mean(1, keepdims=True)) + (0 if dH is None else np.abs(f64(dH)))
    # the mean's 19 U and its own rounding, the products', the difference's, rstd's and the addition's
    err = np.abs(f64(dX) - wx)
    tol = HALF[dtype] * np.abs(wx) + 26 * U * terms * (1 + HALF[dtype])
    assert np.all(err <= tol), float((err - tol).max())
    # dgamma: T / 512 rows a workgroup, then 32 partial rows a wave and 16 waves, two roundings a term
    n = -(-dY.shape[0] // 512) + 32 + 16 + 2
    assert np.all(np.abs(f64(dg) - wg) <= n * U * (np.abs(dy) * xh).sum(0) * (1 + 2 ** -10))


SHAPES = [(1, 1), (2, 7), (3, 64), (5, 65), (4, 127), (4, 128), (3, 129), (17, 1024), (2, 1023), (9, 2048), (4, 2050),
          (3, 2056), (6, 5120), (2, 5121), (3, 8192), (2, 8200), (1, 12288), (2, 16384), (1, 16383), (700, 96), (1030, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward_backward(gpu, dtype, T, H):
    X, R, gamma, dY, dH = data(T, H, dtype, gpu)
    Hs, rstd = check_fwd(X, R, gamma, dtype)
    check_bwd(dY, Hs, gamma, rstd, dH, dtype)
    Hs, rstd = check_fwd(X, None, gamma, dtype, fp8=H % 2 == 0, want_y=H % 2 == 1)
    check_bwd(dY, Hs, gamma, rstd, None, dtype)
    check_fwd(X, R, gamma, dtype, fp8=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_rows_large_and_cancelling_rows(gpu, dtype):
    X, R, gamma, dY, dH = data(5, 520, dtype, gpu)
    X[0] = 0
    R[0] = 0
    X[1] = 3e18  # the square of the sum's terms stays inside fp32
    R[2] = -X[2]  # a sum of zeros
    X[3] *= 1e-12
    R[3] *= 1e-12
    Hs, rstd = check_fwd(X, R, gamma, dtype)
    check_bwd(dY, Hs, gamma, rstd, dH, dtype)


def test_not_finite_stays_in_its_row(gpu):
    X, R, gamma, _, _ = data(4, 300, "bf16", gpu)
    want = sra.rms_norm_fwd(X, gamma, EPS, residual=R, fp8=torch.float8_e4m3fn)
    X2 = X.clone()
    X2[1, 5] = float("nan")
    X2[2, 7] = float("inf")
    Y, H, rstd, F = sra.rms_norm_fwd(X2, gamma, EPS, residual=R, fp8=torch.float8_e4m3fn)
    assert torch.isnan(Y[1]).all() and torch.isnan(Y[2, 7]) and not Y[2, :7].any()
    for got, ref in ((Y, want[0]), (H, want[1]), (F.codes.view(torch.uint8), want[3].codes.view(torch.uint8)), (F.exps, want[3].exps)):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[3], ref[3])
    codes = F.codes.view(torch.uint8)
    assert ((codes[1, :300] & 0x7F) == 0x7F).all() and not codes[1, 300:].any()  # NaN (of either sign), and the filled-up columns stay zeros


@pytest.mark.parametrize("which", ["X", "R"])
def test_sum_in_place(gpu, which):
    X, R, gamma, _, _ = data(33, 1000, "bf16", gpu)
    want = sra.rms_norm_fwd(X, gamma, EPS, residual=R)
    into = X if which == "X" else R
    Y, H, rstd, _ = sra.rms_norm_fwd(X, gamma, EPS, residual=R, H=into)
    assert H is into
    for a, b in zip((Y, H, rstd), want):
        assert np.array_equal(bits(a), bits(b))


@pytest.mark.parametrize("which", ["dY", "dH", "H"])
def test_gradient_in_place(gpu, which):
    X, _, gamma, dY, dH = data(600, 264, "f32", gpu)
    _, H, rstd, _ = sra.rms_norm_fwd(X, gamma, EPS)
    want = sra.rms_norm_bwd(dY, H, gamma, rstd, dH=dH)
    got = sra.rms_norm_bwd(dY, H, gamma, rstd, dH=dH, dX={"dY": dY, "dH": dH, "H": H}[which])
    for a, b in zip(got, want):
        assert np.array_equal(bits(a), bits(b))


def test_empty(gpu):
    z = torch.zeros(0, 64, dtype=torch.bfloat16, device=gpu)
    w = torch.ones(64, dtype=torch.bfloat16, device=gpu)
    Y, _, rstd, F = sra.rms_norm_fwd(z, w, fp8=torch.float8_e4m3fn)
    assert Y.shape == (0, 64) and F.codes.shape == (0, 128) and F.exps.shape == (0, 1)
    _, dg = sra.rms_norm_bwd(z, z, w, torch.zeros(0, device=gpu))
    assert not dg.any()
    n = torch.zeros(3, 0, dtype=torch.bfloat16, device=gpu)
    assert torch.isnan(sra.rms_norm_fwd(n, w[:0])[2]).all()


def test_gradient_by_differences(gpu):
    """Central differences of sum(dY Y) + sum(dH H) in fp32 inputs, evaluated by the float64 oracle."""
    X, R, gamma, dY, dH = data(2, 24, "f32", gpu)
    _, H, rstd, _ = sra.rms_norm_fwd(X, gamma, EPS, residual=R)
    dX, dg = sra.rms_norm_bwd(dY, H, gamma, rstd, dH=dH)
    x, r, ga, dy, dh = (f64(t) for t in (X, R, gamma, dY, dH))

    def loss(x, r, ga):
        y, h, _ = orms.forward(x, r, ga, EPS)
        return float((y * dy).sum() + (h * dh).sum())

    d = 1e-4  # central differences: error d^2 f''' / 6, below 1e-6 here
    for arr, got, at in ((x, f64(dX), (1, 7)), (r, f64(dX), (0, 20)), (ga, f64(dg), (3,))):
        hi, lo = arr.copy(), arr.copy()
        hi[at] += d
        lo[at] -= d
        pick = lambda v: tuple(v if a is arr else a for a in (x, r, ga))
        assert abs((loss(*pick(hi)) - loss(*pick(lo))) / (2 * d) - got[at]) < 1e-4


def test_deterministic(gpu):
    X, _, gamma, dY, _ = data(1500, 1024, "bf16", gpu)
    _, H, rstd, _ = sra.rms_norm_fwd(X, gamma, EPS)
    a, b = (sra.rms_norm_bwd(dY, H, gamma, rstd) for _ in range(2))
    for p, q in zip(a, b):
        assert np.array_equal(bits(p), bits(q))
