"""The example's fine-tuning step: its gradients against the float64 chain of the oracles, each call
compared on the inputs that it actually had (as the step rounds between calls)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import ckpt as ock
from oracle import multi as om
from oracle import nm as onm
from oracle import norm as onorm
from _util import f64, meta_u32

pytestmark = pytest.mark.gpu
U24, BF = 2.0 ** -24, 2.0 ** -8


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "multi_adapter_step.py")
    spec = importlib.util.spec_from_file_location("multi_adapter_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_step(gpu):
    ex = example()
    T, K, N, r, n = 70, 96, 128, 8, 3
    layer = ex.make_layer(K, N, r, n, device=gpu)
    g = torch.Generator().manual_seed(5)
    H = torch.randn(T, K, generator=g).bfloat16().to(gpu)
    dY = torch.randn(T, N, generator=g).bfloat16().to(gpu)
    ids = torch.randint(-1, n, (T,), generator=g).int()
    Y, saved = ex.forward(layer, H, ids.to(gpu))
    grads = ex.backward(layer, dY, saved, weight_grad=True)

    Wd = onm.decompress(f64(layer.Ws.values), meta_u32(layer.Ws.meta), 2, 4, K)
    Pd = onm.decompress(f64(layer.P.values), meta_u32(layer.P.meta), 2, 4, N)
    Wd, Pd = (d[0] if isinstance(d, tuple) else d for d in (Wd, Pd))
    a, b, i = f64(layer.A), f64(layer.B), ids.numpy()
    X = sra.layer_norm_fwd(H, layer.gamma, layer.beta)[0]  # what the step fed to the projection
    x = f64(X)
    wy, _ = om.forward(x, Wd, a, b, i)
    my, _ = om.forward(np.abs(x), np.abs(Wd), np.abs(a), np.abs(b), i)
    assert np.all(np.abs(f64(Y) - wy) <= BF * np.abs(wy) + 2.0 ** -15 * my)

    xv = ock.decode(*ock.encode(x))
    assert np.array_equal(f64(sra.ckpt8_decode(saved[3])), xv)
    u, dy = f64(saved[4]), f64(dY)
    w = om.backward(dy, xv, u, Pd, a, b, i)
    m = om.backward(np.abs(dy), np.abs(xv), np.abs(u), np.abs(Pd), np.abs(a), np.abs(b), i)
    for k in ("dA", "dB"):
        assert np.all(np.abs(f64(grads[k]) - w[k]) <= 160 * U24 * m[k]), k
    D, M = dy.T @ xv, np.abs(dy).T @ np.abs(xv)
    fields = onm.unpack_fields(meta_u32(layer.Ws.meta), K // 2)
    col = (np.arange(K // 2) // 2) * 4 + fields
    dw, mw = np.take_along_axis(D, col, 1), np.take_along_axis(M, col, 1)
    assert np.all(np.abs(f64(grads["dW"]) - dw) <= BF * np.abs(dw) + 70 * U24 * mw)

    dX = sra.multi_lora_bwd(layer.P, dY, saved[3], saved[4], layer.A, layer.B, ids.to(gpu))["dX"]
    wx, wg, wb = onorm.backward(f64(dX), f64(H), f64(layer.gamma), f64(saved[1]), f64(saved[2]))
    xh = (f64(H) - f64(saved[1])[:, None]) * f64(saved[2])[:, None]
    gg = np.abs(f64(dX) * f64(layer.gamma))
    terms = f64(saved[2])[:, None] * (gg + gg.mean(1, keepdims=True) + np.abs(xh) * (gg * np.abs(xh)).mean(1, keepdims=True))
    assert np.all(np.abs(f64(grads["dH"]) - wx) <= BF * np.abs(wx) + 80 * U24 * terms)
    assert np.all(np.abs(f64(grads["dgamma"]) - wg) <= 130 * U24 * (np.abs(f64(dX)) * (np.abs(xh) + 2 * U24)).sum(0))
    assert np.all(np.abs(f64(grads["dbeta"]) - wb) <= 130 * U24 * np.abs(f64(dX)).sum(0))
