"""Layer norm on the GPU against the float64 oracle.

Tolerances count roundings: fp32 sums of H (or T) terms in trees of at most 64 (128) steps, each
half a unit in the last place (2^-24), relative to the magnitudes that are added, and half a step
of the output's type (bf16 2^-8, fp32 2^-24) for its one rounding.
"""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import ckpt as ock
from oracle import norm as onorm
from _util import bits, f64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24
EPS = 1e-5


def data(T, H, dtype, gpu, shift=0.25):
    g = torch.Generator().manual_seed(T * 977 + H)
    t = lambda *s, sd=1.0, m=0.0: (torch.randn(*s, generator=g) * sd + m).to(DT[dtype]).to(gpu)
    return t(T, H, m=shift), t(H, sd=0.1, m=1.0), t(H, sd=0.1), t(T, H)


def check_fwd(X, gamma, beta, dtype, ckpt=False):
    Y, mean, rstd, c = sra.layer_norm_fwd(X, gamma, beta, EPS, ckpt=ckpt)
    x, ga, be = f64(X), f64(gamma), f64(beta)
    y, mu, rs = onorm.forward(x, ga, be, EPS)
    amean = np.abs(x).mean(axis=1)
    assert np.all(np.abs(f64(mean) - mu) <= 64 * U * amean)
    # the variance's relative error: 64 steps on its terms, plus twice the mean's error over the deviation
    dev = np.sqrt(1 / rs ** 2)
    tol_rs = rs * (64 * U + (64 * U * amean / dev) ** 2 + 4 * U)
    assert np.all(np.abs(f64(rstd) - rs) <= tol_rs + 64 * U * rs)
    terms = np.abs(y - be) + (amean * rs)[:, None] * np.abs(ga) + np.abs(be)
    tol = HALF[dtype] * np.abs(y) + (130 * U) * terms * (1 + HALF[dtype])
    err = np.abs(f64(Y) - y)
    assert np.all(err <= tol), float((err - tol).max())
    if ckpt:
        codes, exps = ock.encode(f64(Y))
        assert np.array_equal(c.codes.cpu().numpy(), codes) and np.array_equal(c.exps.cpu().numpy(), exps)
    return Y, mean, rstd


def check_bwd(dY, X, gamma, mean, rstd, dtype):
    dX, dg, db = sra.layer_norm_bwd(dY, X, gamma, mean, rstd)
    dy, x, ga, mu, rs = f64(dY), f64(X), f64(gamma), f64(mean), f64(rstd)
    wx, wg, wb = onorm.backward(dy, x, ga, mu, rs)
    xh = np.abs((x - mu[:, None]) * rs[:, None]) + U * (np.abs(x) + np.abs(mu[:, None])) * rs[:, None]
    g = np.abs(dy * ga)
    terms = rs[:, None] * (g + g.mean(1, keepdims=True) + xh * (g * xh).mean(1, keepdims=True))
    tol = HALF[dtype] * np.abs(wx) + 72 * U * terms * (1 + HALF[dtype])
    err = np.abs(f64(dX) - wx)
    assert np.all(err <= tol), float((err - tol).max())
    assert np.all(np.abs(f64(dg) - wg) <= 128 * U * (np.abs(dy) * xh).sum(0))
    assert np.all(np.abs(f64(db) - wb) <= 128 * U * np.abs(dy).sum(0))


SHAPES = [(1, 1), (2, 7), (3, 64), (5, 65), (17, 1024), (2, 1023), (9, 2048), (4, 2050), (3, 2056), (6, 5120), (2, 5121),
          (3, 8192), (2, 8200), (1, 12288), (2, 16384), (1, 16383), (700, 96), (1030, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward_backward(gpu, dtype, T, H):
    X, gamma, beta, dY = data(T, H, dtype, gpu)
    _, mean, rstd = check_fwd(X, gamma, beta, dtype, ckpt=H % 3 != 0)
    check_bwd(dY, X, gamma, mean, rstd, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_constant_and_shifted_rows(gpu, dtype):
    """Rows of one value (no variance) and rows far from zero."""
    X, gamma, beta, dY = data(4, 520, dtype, gpu)
    X[0] = 0.0
    X[1] = 3.0
    X[2] += 100.0
    _, mean, rstd = check_fwd(X, gamma, beta, dtype)
    check_bwd(dY, X, gamma, mean, rstd, dtype)


def test_empty(gpu):
    z = torch.zeros(0, 64, dtype=torch.bfloat16, device=gpu)
    w = torch.ones(64, dtype=torch.bfloat16, device=gpu)
    e = torch.zeros(0, device=gpu)
    assert sra.layer_norm_fwd(z, w, w)[0].shape == (0, 64)
    _, dg, db = sra.layer_norm_bwd(z, z, w, e, e)
    assert not dg.any() and not db.any()


def test_nan_row_stays_in_its_row(gpu):
    X, gamma, beta, _ = data(3, 128, "bf16", gpu)
    want = sra.layer_norm_fwd(X, gamma, beta)[0]
    X2 = X.clone()
    X2[1, 5] = float("nan")
    got = sra.layer_norm_fwd(X2, gamma, beta)[0]
    assert torch.isnan(got[1]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_gradient_by_differences(gpu):
    """Central differences of sum(dY * Y) in fp32 inputs, evaluated by the float64 oracle."""
    X, gamma, beta, dY = data(2, 24, "f32", gpu)
    _, mean, rstd, _ = sra.layer_norm_fwd(X, gamma, beta, EPS)
    dX, dg, db = sra.layer_norm_bwd(dY, X, gamma, mean, rstd)
    x, ga, be, dy = (f64(t) for t in (X, gamma, beta, dY))
    loss = lambda x, ga, be: float((onorm.forward(x, ga, be, EPS)[0] * dy).sum())
    h = 1e-4  # central differences: error h^2 f''' / 6, below 1e-6 here
    for arr, got, at in ((x, f64(dX), (1, 7)), (ga, f64(dg), (3,)), (be, f64(db), (11,))):
        hi, lo = arr.copy(), arr.copy()
        hi[at] += h
        lo[at] -= h
        pick = lambda v: tuple(v if a is arr else a for a in (x, ga, be))
        assert abs((loss(*pick(hi)) - loss(*pick(lo))) / (2 * h) - got[at]) < 1e-4


def test_deterministic(gpu):
    X, gamma, beta, dY = data(1500, 1024, "bf16", gpu)
    _, mean, rstd, _ = sra.layer_norm_fwd(X, gamma, beta)
    a, b = (sra.layer_norm_bwd(dY, X, gamma, mean, rstd) for _ in range(2))
    for p, q in zip(a, b):
        assert np.array_equal(bits(p), bits(q))
