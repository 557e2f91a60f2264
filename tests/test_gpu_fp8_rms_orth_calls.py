"""How the root-mean-square norm, 8-bit floating point and Newton-Schulz calls are made: captured into a graph and
replayed, on two streams at once, on buffers of the caller, and with arguments they refuse."""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from sparse_rank_adapter_amd._abi import SraError

pytestmark = pytest.mark.gpu


class Step:
    """The calls of one step on buffers of its own; run() fills `out` from `X`, `R`, `W` and `G`."""

    def __init__(self, gpu, T, K, N, seed):
        g = torch.Generator().manual_seed(seed)
        t = lambda *s: torch.randn(*s, generator=g).bfloat16().to(gpu)
        self.X, self.R, self.W, self.gamma = t(T, K), t(T, K), t(N, K), t(K)
        self.G = torch.randn(2, 40, K, generator=g).to(gpu)
        self.G2 = torch.randn(2, 100, 130, generator=g).to(gpu)

    def run(self):
        Y, H, rstd, Y8 = sra.rms_norm_fwd(self.X, self.gamma, residual=self.R, fp8=torch.float8_e4m3fn)
        W8, W8t = sra.fp8_encode_pair(self.W, block_rows=128)
        up = sra.fp8_matmul(Y8, W8)
        d8, d8t = sra.fp8_encode_pair(up, torch.float8_e5m2)
        dY = sra.fp8_matmul(d8, W8t)
        dW = sra.fp8_matmul(d8t, sra.fp8_encode_t(Y), out_dtype=torch.float32)
        dX, dg = sra.rms_norm_bwd(dY, H, self.gamma, rstd, dH=self.R)
        return [Y, H, rstd, up, dY, dW, dX, dg, sra.fp8_decode(Y8), sra.orthogonalize(self.G), sra.orthogonalize(self.G2)]

    def change(self, k):
        for i, t in enumerate((self.X, self.R, self.W, self.G, self.G2)):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(100 * k + i)).to(t.dtype))


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T,K,N", [(9, 200, 300), (70, 1200, 500), (300, 264, 1100)])
def test_captured_and_replayed(gpu, T, K, N):
    s = Step(gpu, T, K, N, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.run()
    for k in range(4):
        s.change(k)
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        want = s.run()  # eager work between the replays
        torch.cuda.synchronize()
        assert same(got, want), k


def test_two_graphs_and_eager_calls_in_turn(gpu):
    steps = [Step(gpu, 50, 300, 400, 2), Step(gpu, 130, 140, 260, 3)]
    graphs, outs = [], []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run())
        graphs.append(g)
    want = [[t.clone() for t in s.run()] for s in steps]
    for _ in range(3):
        for g in graphs:
            g.replay()
        for s in steps:
            s.run()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert same(o, w)


def test_two_streams_at_once(gpu):
    steps = [Step(gpu, 260, 512, 700, 4), Step(gpu, 33, 900, 640, 5)]
    want = [[t.clone() for t in s.run()] for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [None, None]
    for _ in range(5):
        for i, (s, st) in enumerate(zip(steps, streams)):
            with torch.cuda.stream(st):
                got[i] = s.run()
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert same(o, w)


def test_refused_arguments(gpu):
    X = torch.zeros(8, 256, dtype=torch.bfloat16, device=gpu)
    gamma = torch.ones(256, dtype=torch.bfloat16, device=gpu)
    flat = torch.zeros(8 * 256 + 8, dtype=torch.bfloat16, device=gpu)
    off = flat[4:4 + 8 * 256].view(8, 256)  # 8 bytes off a 16-byte boundary
    F = sra.fp8_encode(X)
    for call, err in (
            (lambda: sra.rms_norm_fwd(X[:, :128], gamma[:128]), ValueError), (lambda: sra.rms_norm_fwd(off, gamma), SraError),
            (lambda: sra.rms_norm_fwd(X, gamma.float()), ValueError), (lambda: sra.rms_norm_fwd(X, gamma, residual=X[:4]), ValueError),
            (lambda: sra.rms_norm_fwd(X, gamma, H=X), ValueError), (lambda: sra.rms_norm_fwd(X, gamma, want_y=False), ValueError),
            (lambda: sra.rms_norm_fwd(X, gamma, fp8=torch.float8_e5m2), ValueError), (lambda: sra.rms_norm_fwd(X, gamma, eps=-1.0), SraError),
            (lambda: sra.rms_norm_fwd(X, gamma, fp8=sra.fp8_encode(X, block_rows=128)), ValueError),
            (lambda: sra.rms_norm_bwd(X, X, gamma, torch.zeros(7, device=gpu)), ValueError),
            (lambda: sra.fp8_encode(off), SraError), (lambda: sra.fp8_encode(X, torch.bfloat16), ValueError),
            (lambda: sra.fp8_encode(X, block_rows=2), ValueError), (lambda: sra.fp8_encode(X, out=sra.fp8_encode(X, torch.float8_e5m2)), ValueError),
            (lambda: sra.fp8_decode(F, torch.float16), ValueError), (lambda: sra.fp8_matmul(F, sra.fp8_encode(X[:, :200].contiguous())), ValueError),
            (lambda: sra.fp8_matmul(F, F, out=torch.zeros(8, 9, device=gpu)), ValueError),
            (lambda: sra.fp8_matmul(F, F, out_dtype=torch.float16), ValueError),
            (lambda: sra.orthogonalize(torch.zeros(2, 257, 300, device=gpu)), SraError), (lambda: sra.orthogonalize(X, steps=0), SraError),
            (lambda: sra.orthogonalize(X, out=X), SraError), (lambda: sra.orthogonalize(X[:, ::2]), ValueError)):
        with pytest.raises(err):
            call()


def test_given_buffers_are_the_ones_filled(gpu):
    X = torch.randn(40, 300, device=gpu).bfloat16()
    gamma = torch.ones(300, dtype=torch.bfloat16, device=gpu)
    Y, H = torch.empty_like(X), torch.empty_like(X)
    F = sra.fp8_encode(X)
    y, h, rstd, f = sra.rms_norm_fwd(X, gamma, residual=X, fp8=F, Y=Y, H=H)
    assert y is Y and h is H and f is F
    want = sra.rms_norm_fwd(X, gamma, residual=X, fp8=torch.float8_e4m3fn)
    assert same([y, h, rstd, f.codes.view(torch.uint8), f.exps], [*want[:3], want[3].codes.view(torch.uint8), want[3].exps])
    dX, ws = torch.empty_like(X), torch.empty(1 << 20, dtype=torch.uint8, device=gpu)
    assert sra.rms_norm_bwd(X, H, gamma, rstd, dX=dX, ws=ws)[0] is dX
    out = torch.empty(40, 40, device=gpu)
    assert sra.fp8_matmul(F, F, out=out) is out
