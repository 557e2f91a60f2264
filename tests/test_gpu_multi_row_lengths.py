"""Many adapters beside projections whose output has any length: P of any number of rows K in the backward,
Ws of any number of rows N in the forward, against the float64 oracle.

Tolerances as in test_gpu_multi: n fp32 additions are off by at most n 2^-24 of the sum of magnitudes, two
bf16 parts of U or dU by 2^-16 of each product, a bf16 output by half a step, 2^-8.
"""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import ckpt as ock
from oracle import multi as om
from _util import bits, f64
from test_gpu_multi import BF, U24, close, make_ids, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,r,n", [(1, 8, 2), (16, 40, 3), (40, 8, 4), (75, 130, 3), (300, 24, 5), (300, 64, 5)])
@pytest.mark.parametrize("K", [1, 4, 7, 8, 20, 24, 40, 72, 100, 257])
def test_backward(gpu, K, T, r, n):
    N = 96
    g = torch.Generator().manual_seed(1000 * K + T + r)
    X = torch.randn(T, K, generator=g).bfloat16().to(gpu)
    dY = torch.randn(T, N, generator=g).bfloat16().to(gpu)
    A = (torch.randn(n, r, K, generator=g) * 0.05).bfloat16().to(gpu)
    B = (torch.randn(n, N, r, generator=g) * 0.05).bfloat16().to(gpu)
    ids = make_ids("mixed", T, n, g)
    P, Pd = weight(K, N, 2, 4, g, gpu)
    x, dy, a, b, idn = f64(X), f64(dY), f64(A), f64(B), ids.numpy()
    _, wu = om.forward(x, np.zeros((N, K)), a, b, idn)
    U = torch.from_numpy(wu).float().to(gpu)
    u = f64(U)
    kept = sra.ckpt8_encode(X)
    for name, xin, xv in (("bf16", X, x), ("ckpt", kept, ock.decode(*ock.encode(x)))):
        got = sra.multi_lora_bwd(P, dY, xin, U, A, B, ids.to(gpu), want_du=True)
        want = om.backward(dy, xv, u, Pd, a, b, idn)
        mag = om.backward(np.abs(dy), np.abs(xv), np.abs(u), np.abs(Pd), np.abs(a), np.abs(b), idn)
        close("dU", f64(got["dU"]), want["dU"], 40 * U24 * mag["dU"])
        steps = N // 16 + r + 64
        close("dX", f64(got["dX"]), want["dX"], BF * np.abs(want["dX"]) + (steps * U24 + 2.0 ** -16) * mag["dX"])
        gsteps = 3 * (T // 32 + 2) + 96 + 40
        close("dA", f64(got["dA"]), want["dA"], gsteps * U24 * mag["dA"])
        close("dB", f64(got["dB"]), want["dB"], gsteps * U24 * mag["dB"])
    dec = sra.multi_lora_bwd(P, dY, sra.ckpt8_decode(kept), U, A, B, ids.to(gpu))
    for key in ("dX", "dA", "dB"):
        assert np.array_equal(bits(dec[key]), bits(got[key])), key
    # U recomputed from such rows, too: its own error, of at most 40 2^-24 of the magnitudes, enters dB
    own = sra.multi_lora_bwd(P, dY, X, None, A, B, ids.to(gpu), dx=False, da=False)["dB"]
    _, mu = om.forward(np.abs(x), np.zeros((N, K)), np.abs(a), np.abs(b), idn)
    mag = om.backward(np.abs(dy), np.abs(x), mu, np.abs(Pd), np.abs(a), np.abs(b), idn)
    close("dB from X", f64(own), want["dB"], (gsteps + 41) * U24 * mag["dB"])


@pytest.mark.parametrize("T,r", [(3, 8), (16, 10), (40, 16), (300, 40)])
@pytest.mark.parametrize("N", [1, 20, 43, 200])
def test_forward(gpu, N, T, r):
    K, n = 128, 3
    g = torch.Generator().manual_seed(1000 * N + T)
    X = torch.randn(T, K, generator=g).bfloat16().to(gpu)
    A = (torch.randn(n, r, K, generator=g) * 0.05).bfloat16().to(gpu)
    B = (torch.randn(n, N, r, generator=g) * 0.05).bfloat16().to(gpu)
    ids = make_ids("mixed", T, n, g)
    S, Wd = weight(N, K, 2, 4, g, gpu)
    Y, U = sra.multi_lora_fwd(S, X, A, B, ids.to(gpu))
    x, a, b = f64(X), f64(A), f64(B)
    wy, wu = om.forward(x, Wd, a, b, ids.numpy())
    sy, su = om.forward(np.abs(x), np.abs(Wd), np.abs(a), np.abs(b), ids.numpy())
    close("U", f64(U), wu, 40 * U24 * su)
    close("Y", f64(Y), wy, BF * np.abs(wy) + ((K // 16 + r + 64) * U24 + 2.0 ** -16) * sy)
