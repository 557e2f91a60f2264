"""Newton-Schulz steps on the GPU against the float64 oracle.

Everything but the last rounding (half a step of the type: bf16 2^-8, fp32 2^-24) is fp64.  The Gram matrix is off by at most
L 2^-53 (its trace is 1) and each of the d x d products by d 2^-53; the steps multiply that by at most a^(2 steps) |b| / a
(a small singular value grows by a a step, its square by a^2): 2.4e5 with five steps of the default coefficients.
"""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import orth
from _util import bits, f64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
ABC, EPS = (3.4445, -4.7750, 2.0315), 1e-7
GROW = 3.4445 ** 10 * 4.775 / 3.4445


def data(n, R, C, dtype, gpu, decades=2.0):
    """Some strong directions and noise in all of them, as a gradient has."""
    g = torch.Generator().manual_seed(n * 7 + R * 1009 + C)
    k = min(R, C, 8)
    G = (torch.randn(n, R, k, generator=g) * torch.logspace(0, -decades, k)) @ torch.randn(n, k, C, generator=g)
    return (1e-3 * (G + 10 ** -decades * torch.randn(n, R, C, generator=g))).to(DT[dtype]).to(gpu)


def check(G, dtype, steps=5, abc=ABC, eps=EPS, grow=GROW):
    got = sra.orthogonalize(G, steps=steps, coeffs=abc, eps=eps)
    assert got.shape == G.shape and got.dtype == G.dtype
    g, o = f64(G), f64(got)
    if g.ndim == 2:
        g, o = g[None], o[None]
    d, L = sorted(g.shape[1:])
    for x, y in zip(g, o):
        want = orth.orthogonalize(x, steps, abc, eps)
        err = np.abs(y - want)
        tol = HALF[dtype] * (1 + 2 ** -20) * np.abs(want) + (L + 4 * steps * d) * 2.0 ** -53 * grow
        assert np.all(err <= tol), (float((err - tol).max()), float(np.abs(want).max()))


SHAPES = [(1, 1, 1), (2, 1, 50), (3, 3, 17), (1, 4, 4), (2, 15, 33), (5, 16, 1024), (2, 16, 999), (3, 17, 64), (2, 31, 500),
          (2, 32, 257), (2, 33, 300), (2, 48, 130), (2, 64, 640), (1, 64, 64), (2, 65, 200), (1, 100, 1001), (2, 128, 512),
          (1, 128, 2050), (1, 129, 300), (1, 200, 444), (1, 256, 256), (2, 256, 1000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,L", SHAPES)
def test_wide_and_tall(gpu, dtype, n, d, L):
    check(data(n, d, L, dtype, gpu), dtype)
    check(data(n, L, d, dtype, gpu), dtype)


@pytest.mark.parametrize("d", [16, 64, 96])
@pytest.mark.parametrize("steps", [1, 2, 7])
def test_steps_and_coefficients(gpu, d, steps):
    check(data(2, d, 300, "f32", gpu), "f32", steps=steps, grow=GROW ** (steps / 5) + 10)
    check(data(2, 300, d, "f32", gpu), "f32", steps=steps, abc=(1.5, -0.5, 0.0), grow=1.5 ** (2 * steps))


@pytest.mark.parametrize("d", [16, 64, 128])
def test_orthonormal_after_many_steps(gpu, d):
    G = torch.randn(d, 700, generator=torch.Generator().manual_seed(1)).to(gpu)
    O = f64(sra.orthogonalize(G, steps=40, coeffs=(1.5, -0.5, 0.0)))
    # the steps converge; what is left is the output's rounding, 2^-24 of each element
    assert np.abs(O @ O.T - np.eye(d)).max() <= 2 * 2.0 ** -24 * 1.01


@pytest.mark.parametrize("d,L", [(8, 100), (64, 300), (100, 400)])
def test_far_singular_values(gpu, d, L):
    """Directions four decades below the strongest, where fp32 steps are off by 1e-5 and more."""
    check(data(2, d, L, "f32", gpu, decades=4.0), "f32")


@pytest.mark.parametrize("d", [16, 64, 128])
def test_sizes_zero_and_not_finite(gpu, d):
    G = data(6, d, 200, "f32", gpu)
    want = sra.orthogonalize(G)
    G[1] *= 2.0 ** 100  # the sum of squares is past fp32
    G[2] = 0
    G[3, 0, 5] = float("nan")
    G[4, 1, 6] = float("inf")
    got = sra.orthogonalize(G)
    assert np.array_equal(bits(got[0]), bits(want[0])) and np.array_equal(bits(got[5]), bits(want[5]))
    assert torch.isnan(got[3]).all() and torch.isnan(got[4]).all()
    assert not got[2].any()
    # as if eps were 2^-100 of itself
    check(G[1].contiguous(), "f32")


def test_empty_two_dimensions_and_given_buffers(gpu):
    for s in ((0, 4, 8), (3, 0, 8), (3, 8, 0), (0, 5)):
        assert sra.orthogonalize(torch.zeros(s, device=gpu)).shape == s
    G = data(3, 40, 500, "f32", gpu)
    want = sra.orthogonalize(G)
    ws = torch.full((sra.orthogonalize_workspace(3, 40, 500) + 64,), 0xFF, dtype=torch.uint8, device=gpu)
    out = torch.empty_like(G)
    for _ in range(3):
        assert sra.orthogonalize(G, out=out, ws=ws) is out
        assert np.array_equal(bits(out), bits(want))
