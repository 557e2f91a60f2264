"""Activations of more than 2^31 elements (4 GiB): offsets of the many-adapter, checkpoint and layer norm
calls.  Most tokens are zero; the ones that count lie at both ends and around the 2^31st element.

Tolerances as in the tests of the single calls: a token's sums have the same number of roundings here, and zero
tokens add none to the gradients.
"""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import multi as om
from oracle import nm as onm
from _util import bits, f64

pytestmark = pytest.mark.gpu
U24, BF = 2.0 ** -24, 2.0 ** -8
T, WIDE = 70001, 40960
EDGE = 2 ** 31 // WIDE
ROWS = [0, 1, 31, 32, 4097, EDGE - 1, EDGE, EDGE + 1, T - 33, T - 2, T - 1]


def weight(rows, cols, g, gpu):
    W = (torch.randn(rows, cols, generator=g) * 0.05).bfloat16()
    return sra.compress(W.to(gpu)), np.where(onm.compress(f64(W), 2, 4)[2], f64(W), 0.0)


def close(name, got, want, tol):
    assert np.all(np.abs(got - want) <= tol), (name, float((np.abs(got - want) - tol).max()))


@pytest.mark.parametrize("r", [8, 40])
def test_multi_lora(gpu, r):
    g = torch.Generator().manual_seed(r)
    K, N, n = 64, WIDE, 3
    S, Wd = weight(N, K, g, gpu)
    P, Pd = weight(K, N, g, gpu)
    A = (torch.randn(n, r, K, generator=g) * 0.05).bfloat16()
    B = (torch.randn(n, N, r, generator=g) * 0.05).bfloat16()
    ids = torch.randint(-1, n, (T,), generator=g).int()
    x, dy = torch.randn(len(ROWS), K, generator=g).bfloat16(), torch.randn(len(ROWS), N, generator=g).bfloat16()
    rows = torch.tensor(ROWS)
    X = torch.zeros(T, K, dtype=torch.bfloat16)
    X[rows] = x
    X = X.to(gpu)
    dY = torch.zeros(T, N, dtype=torch.bfloat16, device=gpu)
    dY[rows.to(gpu)] = dy.to(gpu)
    a, b, idn = f64(A), f64(B), ids[rows].numpy()
    A, B, ids = A.to(gpu), B.to(gpu), ids.to(gpu)
    pick = rows.to(gpu)

    Y, U = sra.multi_lora_fwd(S, X, A, B, ids)
    wy, wu = om.forward(f64(x), Wd, a, b, idn)
    sy, su = om.forward(np.abs(f64(x)), np.abs(Wd), np.abs(a), np.abs(b), idn)
    close("U", f64(U[pick]), wu, 40 * U24 * su)
    close("Y", f64(Y[pick]), wy, BF * np.abs(wy) + ((K // 16 + r + 64) * U24 + 2.0 ** -16) * sy)
    assert int(torch.count_nonzero(Y.any(1))) <= len(ROWS)
    del Y

    u = f64(U[pick])
    want = om.backward(f64(dy), f64(x), u, Pd, a, b, idn)
    mag = om.backward(np.abs(f64(dy)), np.abs(f64(x)), np.abs(u), np.abs(Pd), np.abs(a), np.abs(b), idn)
    got = sra.multi_lora_bwd(P, dY, X, U, A, B, ids, want_du=True)
    close("dU", f64(got["dU"][pick]), want["dU"], 40 * U24 * mag["dU"])
    close("dX", f64(got["dX"][pick]), want["dX"],
          BF * np.abs(want["dX"]) + ((N // 16 + r + 64) * U24 + 2.0 ** -16) * mag["dX"])
    steps = 3 * (T // 32 + 2) + 96 + 40
    close("dA", f64(got["dA"]), want["dA"], steps * U24 * mag["dA"])
    close("dB", f64(got["dB"]), want["dB"], steps * U24 * mag["dB"])
    # dX = 0 where dY is
    assert int(torch.count_nonzero(got["dX"].any(1))) <= len(ROWS)


@pytest.mark.parametrize("r", [8, 40])
def test_wide_input(gpu, r):
    """The layer's input is the long operand: dA, from bf16 and from its checkpoint, and the forward."""
    g = torch.Generator().manual_seed(100 + r)
    K, N, n = WIDE, 64, 2
    S, Wd = weight(N, K, g, gpu)
    A = (torch.randn(n, r, K, generator=g) * 0.05).bfloat16()
    B = (torch.randn(n, N, r, generator=g) * 0.05).bfloat16()
    ids = torch.randint(-1, n, (T,), generator=g).int()
    P, _ = weight(K, N, g, gpu)
    x, dy = torch.randn(len(ROWS), K, generator=g).bfloat16(), torch.randn(len(ROWS), N, generator=g).bfloat16()
    rows = torch.tensor(ROWS)
    pick = rows.to(gpu)
    X = torch.zeros(T, K, dtype=torch.bfloat16, device=gpu)
    X[pick] = x.to(gpu)
    dY = torch.zeros(T, N, dtype=torch.bfloat16)
    dY[rows] = dy
    a, b, idn = f64(A), f64(B), ids[rows].numpy()
    A, B, ids, dY = A.to(gpu), B.to(gpu), ids.to(gpu), dY.to(gpu)
    Y, U = sra.multi_lora_fwd(S, X, A, B, ids)
    wy, wu = om.forward(f64(x), Wd, a, b, idn)
    sy, su = om.forward(np.abs(f64(x)), np.abs(Wd), np.abs(a), np.abs(b), idn)
    close("U", f64(U[pick]), wu, 40 * U24 * su)
    close("Y", f64(Y[pick]), wy, BF * np.abs(wy) + ((K // 16 + r + 64) * U24 + 2.0 ** -16) * sy)

    kept = sra.ckpt8_encode(X)
    part = sra.ckpt8_encode(x.to(gpu))
    assert torch.equal(kept.codes[pick], part.codes) and torch.equal(kept.exps[pick], part.exps)
    for name, xin, xv in (("bf16", X, f64(x)), ("ckpt", kept, f64(sra.ckpt8_decode(part)))):
        want = om.backward(f64(dy), xv, wu, np.zeros((K, N)), a, b, idn)
        mag = om.backward(np.abs(f64(dy)), np.abs(xv), np.abs(wu), np.zeros((K, N)), np.abs(a), np.abs(b), idn)
        got = sra.multi_lora_bwd(P, dY, xin, U, A, B, ids, dx=False, db=False)
        close(name, f64(got["dA"]), want["dA"], (3 * (T // 32 + 2) + 96 + 40) * U24 * mag["dA"])
    back = sra.ckpt8_decode(kept)
    assert np.array_equal(bits(back[pick]), bits(sra.ckpt8_decode(part)))


def test_layer_norm(gpu):
    g = torch.Generator().manual_seed(7)
    T, WIDE = 140001, 16384
    ROWS = [0, 1, 2 ** 31 // WIDE - 1, 2 ** 31 // WIDE, 2 ** 31 // WIDE + 1, T - 2, T - 1]
    x = torch.randn(len(ROWS), WIDE, generator=g).bfloat16().to(gpu)
    dy = torch.randn(len(ROWS), WIDE, generator=g).bfloat16().to(gpu)
    gamma = torch.randn(WIDE, generator=g).bfloat16().to(gpu)
    beta = torch.randn(WIDE, generator=g).bfloat16().to(gpu)
    pick = torch.tensor(ROWS, device=gpu)
    X = torch.ones(T, WIDE, dtype=torch.bfloat16, device=gpu)
    X[pick] = x
    Y, mean, rstd, c = sra.layer_norm_fwd(X, gamma, beta, ckpt=True)
    y1, m1, r1, c1 = sra.layer_norm_fwd(x, gamma, beta, ckpt=True)
    for got, want in ((Y, y1), (mean, m1), (rstd, r1), (c.codes, c1.codes), (c.exps, c1.exps)):
        assert torch.equal(got[pick], want)  # a row's result depends on the row alone
    del Y, c
    dY = torch.zeros(T, WIDE, dtype=torch.bfloat16, device=gpu)
    dY[pick] = dy
    dX, dg, db = sra.layer_norm_bwd(dY, X, gamma, mean, rstd)
    dx1, _, _ = sra.layer_norm_bwd(dy, x, gamma, m1, r1)
    assert np.array_equal(bits(dX[pick]), bits(dx1))
    xh = (f64(x) - f64(m1)[:, None]) * f64(r1)[:, None]
    d = f64(dy)
    # fp32 sums of at most len(ROWS) terms that are not zero, each term three roundings
    close("dgamma", f64(dg), (d * xh).sum(0), (len(ROWS) + 4) * U24 * np.abs(d * (np.abs(xh) + np.abs(f64(m1) * f64(r1))[:, None])).sum(0))
    close("dbeta", f64(db), d.sum(0), (len(ROWS) + 1) * U24 * np.abs(d).sum(0))
