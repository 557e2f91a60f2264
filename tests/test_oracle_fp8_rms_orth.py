"""Pins of the 8-bit floating point, root-mean-square norm and Newton-Schulz oracles (CPU)."""
import numpy as np
import pytest
import torch

from oracle import fp8, orth, rms

DT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_code_values_are_the_types(kind):
    want = torch.arange(256, dtype=torch.uint8).view(DT[kind]).double().numpy()
    assert np.array_equal(fp8.values(kind), want, equal_nan=True)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_rounding_is_to_nearest_even(kind):
    v = fp8.values(kind)[:fp8.KINDS[kind][3] + 1]
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), -v, -mid])
    x = x[x == x.astype(np.float32)]  # what the other converter takes
    want = torch.from_numpy(x.astype(np.float32)).to(DT[kind]).view(torch.uint8).numpy()
    assert np.array_equal(fp8.nearest(x, kind), want)


@pytest.mark.parametrize("kind,lim", [("e4m3", 448.0), ("e5m2", 57344.0)])
def test_scale_is_the_smallest_that_fits(kind, lim):
    rng = np.random.default_rng(0)
    X = rng.standard_normal((40, 200)) * 10.0 ** rng.uniform(-20, 20, (40, 1))
    X[0] = 0
    X[1] = 0
    X[1, 0] = lim * 8
    codes, exps = fp8.encode(X, kind)
    for j, at in enumerate((slice(0, 128), slice(128, 200))):
        top = np.abs(X[:, at]).max(1)
        s = 2.0 ** (exps[:, j].astype(int) - 127)
        assert np.all(top <= lim * s) and np.all((top > lim * s / 2) | (exps[:, j] == 1))
    assert exps[1, 0] == 130 and exps[0, 0] == 1
    got = fp8.decode(codes, exps, kind, 200)
    half = 2.0 ** -4 if kind == "e4m3" else 2.0 ** -3
    low = 2.0 ** -10 if kind == "e4m3" else 2.0 ** -17
    step = np.repeat(2.0 ** (exps.astype(int) - 127), 128, axis=1)[:, :200]
    assert np.all(np.abs(got - X) <= np.maximum(half * np.abs(X), low * step))


def test_blocks_of_128_rows_transpose():
    X = np.random.default_rng(1).standard_normal((150, 270))
    c, e = fp8.encode(X, "e4m3", 128)
    ct, et = fp8.encode(X.T, "e4m3", 128)
    assert np.array_equal(e.T, et) and np.array_equal(c[:, :270].T, ct[:, :150])


def test_rms_gradient_is_autograds():
    t = lambda *s: torch.randn(*s, dtype=torch.float64)
    torch.manual_seed(0)
    X, R, gamma, dY, dH = t(5, 9), t(5, 9), t(9), t(5, 9), t(5, 9)
    for v in (X, R, gamma):
        v.requires_grad_()
    H = X + R
    Y = H * torch.rsqrt(H.square().mean(1, keepdim=True) + 1e-3) * gamma
    ((Y * dY).sum() + (H * dH).sum()).backward()
    y, h, rstd = rms.forward(*(v.detach().numpy() for v in (X, R, gamma)), 1e-3)
    assert np.allclose(y, Y.detach().numpy(), rtol=1e-12)
    dx, dg = rms.backward(dY.numpy(), h, gamma.detach().numpy(), rstd, dH.numpy())
    assert np.allclose(dx, X.grad.numpy(), rtol=1e-10) and np.allclose(dx, R.grad.numpy(), rtol=1e-10)
    assert np.allclose(dg, gamma.grad.numpy(), rtol=1e-10)


@pytest.mark.parametrize("shape", [(6, 40), (40, 6), (7, 7)])
def test_newton_schulz_maps_the_singular_values(shape):
    G = np.random.default_rng(2).standard_normal(shape)
    u, v, w = np.linalg.svd(G, full_matrices=False)
    v = v / np.linalg.norm(G)
    for _ in range(5):
        v = 3.4445 * v - 4.7750 * v ** 3 + 2.0315 * v ** 5
    assert np.allclose(orth.orthogonalize(G, 5, (3.4445, -4.7750, 2.0315), 0.0), (u * v) @ w, atol=1e-10)
    # and with the classical coefficients many steps give orthonormal rows (or columns)
    O = orth.orthogonalize(G, 40, (1.5, -0.5, 0.0), 0.0)
    assert np.allclose(O @ O.T if shape[0] <= shape[1] else O.T @ O, np.eye(min(shape)), atol=1e-8)
