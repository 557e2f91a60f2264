"""Many adapters beside one projection on the GPU against the float64 oracle.

Tolerances count roundings.  Sums of products of bf16 values (exact in fp32) run in fp32 partials:
each addition is off by at most 2^-24 of the partial sum, which the sum of magnitudes S bounds, so n
additions give n 2^-24 S.  U and dU enter the outputs' epilogue as two bf16 parts (2^-16 of each
product) and the adapter gradients as three (2^-24).  Outputs add half a step of their type.
"""
import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import ckpt as ock
from oracle import multi as om
from oracle import nm as onm
from _util import bits, f64

pytestmark = pytest.mark.gpu
U24, BF = 2.0 ** -24, 2.0 ** -8


def weight(rows, cols, n, m, g, gpu):
    """(compressed, dense float64 of its kept entries)"""
    W = (torch.randn(rows, cols, generator=g) * 0.05).bfloat16()
    S = sra.compress(W.to(gpu), n, m)
    mask = onm.compress(f64(W), n, m)[2]
    return S, np.where(mask, f64(W), 0.0)


def make_ids(kind, T, n, g):
    if kind == "one":
        return torch.zeros(T, dtype=torch.int32)
    if kind == "none":
        return torch.full((T,), -1, dtype=torch.int32)
    if kind == "mixed":
        return torch.randint(-1, n, (T,), generator=g).int()
    if kind == "wild":  # ids that name no adapter, from both ends of the range
        v = torch.tensor([-2 ** 31, 2 ** 31 - 1, n, -1, 0, n - 1])
        return v[torch.randint(0, 6, (T,), generator=g)].int()
    cuts = torch.sort(torch.randint(0, T + 1, (max(1, n),), generator=g)).values
    seg = torch.bucketize(torch.arange(T), cuts, right=True)
    return torch.randint(0, n, (n + 1,), generator=g)[seg].int()


def close(name, got, want, tol):
    err = np.abs(got - want)
    assert np.all(err <= tol), (name, float((err - tol).max()), np.unravel_index(np.argmax(err - tol), err.shape))


def run(gpu, T, K, N, r, n, kind, fmt=(2, 4), tiled=False, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * T + K + 3 * N + r)
    X = torch.randn(T, K, generator=g).bfloat16().to(gpu)
    dY = torch.randn(T, N, generator=g).bfloat16().to(gpu)
    A = (torch.randn(n, r, K, generator=g) * 0.05).bfloat16().to(gpu)
    B = (torch.randn(n, N, r, generator=g) * 0.05).bfloat16().to(gpu)
    ids = make_ids(kind, T, n, g)
    S, Wd = weight(N, K, *fmt, g, gpu)
    P, Pd = weight(K, N, *fmt, g, gpu)
    if tiled:
        S, P = sra.nm_tile(S), sra.nm_tile(P)
    di = ids.to(gpu)
    x, dy, a, b, idn = f64(X), f64(dY), f64(A), f64(B), ids.numpy()

    Y, U = sra.multi_lora_fwd(S, X, A, B, di)
    wy, wu = om.forward(x, Wd, a, b, idn)
    ax = np.abs(x)
    _, su = om.forward(ax, np.abs(Wd), np.abs(a), np.abs(b), idn)
    sy, _ = om.forward(ax, np.abs(Wd), np.abs(a), np.abs(b), idn)
    close("U", f64(U), wu, 40 * U24 * su)
    steps = K // 16 + r + 64
    close("Y", f64(Y), wy, BF * np.abs(wy) + (steps * U24 + 2.0 ** -16) * sy)

    u = f64(U)
    kept = sra.ckpt8_encode(X)
    res = {}
    for name, xin in (("bf16", X), ("ckpt", kept)):
        xv = x if name == "bf16" else ock.decode(*ock.encode(x))
        got = sra.multi_lora_bwd(P, dY, xin, U, A, B, di, want_du=True)
        want = om.backward(dy, xv, u, Pd, a, b, idn)
        mag = om.backward(np.abs(dy), np.abs(xv), np.abs(u), np.abs(Pd), np.abs(a), np.abs(b), idn)
        close("dU", f64(got["dU"]), want["dU"], 40 * U24 * mag["dU"])
        steps = N // 16 + r + 64
        close("dX", f64(got["dX"]), want["dX"], BF * np.abs(want["dX"]) + (steps * U24 + 2.0 ** -16) * mag["dX"])
        gsteps = 3 * (T // 32 + 2) + 96 + 40  # three parts a step, 32 products each; dU's own error
        close("dA", f64(got["dA"]), want["dA"], gsteps * U24 * mag["dA"])
        close("dB", f64(got["dB"]), want["dB"], gsteps * U24 * mag["dB"])
        res[name] = got
    # the checkpoint's gradients are those of the decoded values, bit for bit
    dec = sra.multi_lora_bwd(P, dY, sra.ckpt8_decode(kept), U, A, B, di)
    for key in ("dX", "dA", "dB"):
        assert np.array_equal(bits(dec[key]), bits(res["ckpt"][key])), key
    return S, P, X, dY, A, B, di, U, res


KINDS = ["one", "none", "mixed", "wild", "requests"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 3, 16])
def test_few_tokens(gpu, T, kind):
    run(gpu, T, 192, 96, 8, 5, kind)


@pytest.mark.parametrize("r", [1, 3, 8, 16, 24, 32, 40, 64, 100, 128, 136, 256])
def test_ranks(gpu, r):
    run(gpu, 16, 128, 160, r, 3, "mixed")
    run(gpu, 70, 128, 160, r, 3, "requests")
    run(gpu, 300, 128, 192, r, 3, "mixed")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,K,N", [(17, 32, 32), (33, 96, 64), (129, 64, 320), (257, 160, 128), (300, 256, 384)])
def test_shapes(gpu, T, K, N, kind):
    run(gpu, T, K, N, 16, 7, kind)


@pytest.mark.parametrize("T", [1, 16, 17, 130, 600])
@pytest.mark.parametrize("kind", ["mixed", "requests"])
def test_streaming_layout(gpu, T, kind):
    run(gpu, T, 256, 384, 16, 6, kind, tiled=True)


@pytest.mark.parametrize("fmt", [(1, 2), (2, 8)])
@pytest.mark.parametrize("T", [5, 40])
def test_other_patterns(gpu, T, fmt):
    run(gpu, T, 256, 128, 16, 4, "mixed", fmt=fmt)


@pytest.mark.parametrize("T", [4, 50])
def test_2_8_streaming(gpu, T):
    run(gpu, T, 256, 128, 8, 4, "mixed", fmt=(2, 8), tiled=True)


def test_large_tiles(gpu):
    """Token and row counts that take the 256x128 and 256x256 tiles, and a split reduction."""
    run(gpu, 640, 128, 16384, 8, 3, "requests")
    run(gpu, 100, 4096, 128, 16, 9, "mixed")


@pytest.mark.parametrize("kind", ["mixed", "requests"])
@pytest.mark.parametrize("T,K,N,r,n,tiled", [(17, 2048, 128, 16, 12, True), (64, 1024, 256, 40, 30, True),
                                             (50, 768, 640, 4, 35, True), (100, 1600, 128, 8, 9, False),
                                             (28, 544, 160, 128, 18, False), (130, 1056, 96, 10, 3, False)])
def test_split_reduction(gpu, T, K, N, r, n, tiled, kind):
    """Few tiles: the reduction is split and the splits share the adapters (more adapters than splits, and
    fewer), in both layouts, with a short last split, and on the tile of reductions of 64 i + 32."""
    run(gpu, T, K, N, r, n, kind, tiled=tiled)


def test_middle_tiles(gpu):
    """More than 128 tiles of 256 x 128 and fewer than fill the GPU."""
    run(gpu, 1300, 128, 4096, 40, 5, "mixed")


def test_many_adapters(gpu):
    run(gpu, 200, 64, 64, 4, 1023, "mixed")
    run(gpu, 1500, 64, 32, 4, 700, "mixed")


@pytest.mark.parametrize("n", [5, 70])
@pytest.mark.parametrize("kind", ["mixed", "requests"])
def test_long_batches(gpu, n, kind):
    """More tokens than the sort's workgroup keeps in registers."""
    run(gpu, 9001, 64, 32, 4, n, kind)


@pytest.mark.parametrize("T", [32, 33, 34, 64, 100, 255, 256, 257])
@pytest.mark.parametrize("r", [4, 24, 64])
def test_single_tokens_of_many_adapters(gpu, T, r):
    """Batches whose tokens each take an adapter of their own choice: the order of the work, not the results,
    depends on them."""
    run(gpu, T, 128, 96, r, 40, "mixed")
    g = torch.Generator().manual_seed(T)
    S, _ = weight(96, 128, 2, 4, g, gpu)
    X = torch.randn(T, 128, generator=g).bfloat16().to(gpu)
    A = (torch.randn(40, r, 128, generator=g) * 0.05).bfloat16().to(gpu)
    B = (torch.randn(40, 96, r, generator=g) * 0.05).bfloat16().to(gpu)
    ids = make_ids("mixed", T, 40, g).to(gpu)
    Y, U = sra.multi_lora_fwd(S, X, A, B, ids)
    order = torch.argsort(ids, stable=True)
    Ys, Us = sra.multi_lora_fwd(S, X[order].contiguous(), A, B, ids[order].contiguous())
    assert torch.equal(U[order], Us) and torch.equal(Y[order], Ys)


def test_one_adapter_equals_the_layer(gpu):
    """With one adapter for every token, the outputs of the one-adapter layer to rounding."""
    S, P, X, dY, A, B, di, U, res = run(gpu, 96, 128, 64, 8, 1, "one")
    Y1, U1 = sra.sparse_lora_fwd(S, X, A[0].contiguous(), B[0].contiguous())
    assert float((U1 - U).abs().max()) <= 1e-5
    Y, _ = sra.multi_lora_fwd(S, X, A, B, di)
    assert float((Y1.float() - Y.float()).abs().max()) <= 2 ** -7 * float(Y1.float().abs().max())


def test_u_recomputed_and_partial_outputs(gpu):
    S, P, X, dY, A, B, di, U, res = run(gpu, 75, 128, 96, 16, 4, "mixed")
    full = res["bf16"]
    only = sra.multi_lora_bwd(P, dY, X, None, A, B, di, dx=False, da=False)  # U recomputed from X
    assert np.array_equal(bits(only["dB"]), bits(full["dB"])) and "dX" not in only
    kept = sra.ckpt8_encode(X)
    a = sra.multi_lora_bwd(P, dY, kept, None, A, B, di, dx=False, da=False)
    b = sra.multi_lora_bwd(P, dY, sra.ckpt8_decode(kept), None, A, B, di, dx=False, da=False)
    assert np.array_equal(bits(a["dB"]), bits(b["dB"]))
    only = sra.multi_lora_bwd(P, dY, None, U, A, B, di, da=False, db=False)
    assert np.array_equal(bits(only["dX"]), bits(full["dX"]))
    plain = sra.multi_lora_bwd(P, dY, None, U, A, B, di, da=False, db=False, dx_adapter=False)["dX"]
    none = sra.multi_lora_bwd(P, dY, None, U, A, B, torch.full_like(di, -1), da=False, db=False)["dX"]
    assert np.array_equal(bits(plain), bits(none))


def test_empty_batch(gpu):
    g = torch.Generator().manual_seed(3)
    S, _ = weight(64, 96, 2, 4, g, gpu)
    P, _ = weight(96, 64, 2, 4, g, gpu)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=gpu)
    ids = torch.zeros(0, dtype=torch.int32, device=gpu)
    Y, U = sra.multi_lora_fwd(S, z(0, 96), z(2, 4, 96), z(2, 64, 4), ids)
    assert Y.shape == (0, 64) and U.shape == (0, 4)
    out = sra.multi_lora_bwd(P, z(0, 64), z(0, 96), U, z(2, 4, 96), z(2, 64, 4), ids)
    assert not out["dA"].any() and not out["dB"].any()


def test_deterministic_and_other_stream(gpu):
    S, P, X, dY, A, B, di, U, res = run(gpu, 500, 256, 256, 16, 9, "mixed")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        Y2, U2 = sra.multi_lora_fwd(S, X, A, B, di)
        g2 = sra.multi_lora_bwd(P, dY, X, U, A, B, di)
    torch.cuda.current_stream().wait_stream(s)
    Y1, U1 = sra.multi_lora_fwd(S, X, A, B, di)
    assert np.array_equal(bits(Y1), bits(Y2)) and np.array_equal(bits(U1), bits(U2))
    for k in ("dX", "dA", "dB"):
        assert np.array_equal(bits(res["bf16"][k]), bits(g2[k])), k


def test_graph_replay(gpu):
    """A captured forward and backward follow new inputs and new ids on every replay."""
    S, P, X, dY, A, B, di, U, res = run(gpu, 200, 128, 128, 8, 5, "mixed")
    ws_f = torch.empty(1 << 20, dtype=torch.uint8, device=gpu)
    ws_b = torch.empty(8 << 20, dtype=torch.uint8, device=gpu)
    Y, Ub = torch.empty(200, 128, dtype=torch.bfloat16, device=gpu), torch.empty(200, 8, device=gpu)
    out = {k: torch.empty_like(v) for k, v in res["bf16"].items() if k != "dU"}

    def step():
        sra.multi_lora_fwd(S, X, A, B, di, Y=Y, U=Ub, ws=ws_f)
        sra.multi_lora_bwd(P, dY, X, Ub, A, B, di, ws=ws_b, out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        X.copy_(torch.randn_like(X.float()).bfloat16())
        di.copy_(torch.randint(-1, 5, (200,), dtype=torch.int32, device=gpu))
        graph.replay()
        torch.cuda.synchronize()
        got = [Y.clone(), Ub.clone()] + [out[k].clone() for k in sorted(out)]
        Ye, Ue = sra.multi_lora_fwd(S, X, A, B, di)
        ge = sra.multi_lora_bwd(P, dY, X, Ue, A, B, di)
        for p, q in zip(got, [Ye, Ue] + [ge[k] for k in sorted(ge)]):
            assert np.array_equal(bits(p), bits(q))


@pytest.mark.parametrize("T,R,C", [(1, 8, 32), (37, 64, 96), (100, 72, 128), (300, 256, 512)])
@pytest.mark.parametrize("fmt", [(2, 4), (1, 2)])
def test_masked_weight_grad_from_checkpoint(gpu, T, R, C, fmt):
    g = torch.Generator().manual_seed(T + R)
    S, _ = weight(R, C, *fmt, g, gpu)
    dY = torch.randn(T, R, generator=g).bfloat16().to(gpu)
    X = torch.randn(T, C, generator=g).bfloat16().to(gpu)
    kept = sra.ckpt8_encode(X)
    got = sra.masked_weight_grad(S, dY, kept)
    want = sra.masked_weight_grad(S, dY, sra.ckpt8_decode(kept))
    assert np.array_equal(bits(got), bits(want))
    # and the definition: the dense gradient of the decoded values at the stored positions
    xv = ock.decode(*ock.encode(f64(X)))
    D, M = f64(dY).T @ xv, np.abs(f64(dY)).T @ np.abs(xv)
    d = sra.SparseMatrix(S.fmt, S.dtype, S.rows, S.cols, torch.ones_like(S.values), meta=S.meta, n=S.n, m=S.m)
    words = d.meta.cpu().numpy().view(np.uint32)
    i = np.arange(C // S.m * S.n)
    pos = (words[:, i // 16] >> (2 * (i % 16)).astype(np.uint32)) & 3
    col = (i // S.n) * S.m + pos
    w, mag = np.take_along_axis(D, col, 1), np.take_along_axis(M, col, 1)
    assert np.all(np.abs(f64(got) - w) <= BF * np.abs(w) + 70 * U24 * mag)


@pytest.mark.parametrize("T,K,N", [(12, 128, 96), (150, 128, 96), (150, 96, 64), (300, 256, 256)])
def test_one_request_cannot_reach_another(gpu, T, K, N):
    """Infinities and NaN in one adapter, or in one adapter's tokens, leave every other token's results and
    every other adapter's gradients as they were."""
    g = torch.Generator().manual_seed(T + K)
    r, n = 40 if T == 300 else 8, 4
    S, _ = weight(N, K, 2, 4, g, gpu)
    P, _ = weight(K, N, 2, 4, g, gpu)
    X = torch.randn(T, K, generator=g).bfloat16().to(gpu)
    dY = torch.randn(T, N, generator=g).bfloat16().to(gpu)
    A = (torch.randn(n, r, K, generator=g) * 0.05).bfloat16().to(gpu)
    B = (torch.randn(n, N, r, generator=g) * 0.05).bfloat16().to(gpu)
    ids = make_ids("mixed", T, n, g).to(gpu)
    others = ids != 2
    keep = [0, 1, 3]
    Y, U = sra.multi_lora_fwd(S, X, A, B, ids)
    want = sra.multi_lora_bwd(P, dY, X, U, A, B, ids)

    A2, B2 = A.clone(), B.clone()
    A2[2, 1] = float("nan")
    B2[2, ::3] = float("inf")
    Yb, Ub = sra.multi_lora_fwd(S, X, A2, B2, ids)
    got = sra.multi_lora_bwd(P, dY, X, Ub, A2, B2, ids)
    assert torch.equal(Yb[others], Y[others]) and torch.equal(Ub[others], U[others])
    assert not torch.isfinite(Yb[~others]).all()
    assert torch.equal(got["dX"][others], want["dX"][others])
    for k in ("dA", "dB"):
        assert torch.equal(got[k][keep], want[k][keep]), k

    X2, dY2 = X.clone(), dY.clone()
    X2[~others] = float("nan")
    dY2[~others] = float("inf")
    Yb, Ub = sra.multi_lora_fwd(S, X2, A, B, ids)
    got = sra.multi_lora_bwd(P, dY2, X2, Ub, A, B, ids)
    assert torch.equal(Yb[others], Y[others]) and torch.equal(Ub[others], U[others])
    assert torch.equal(got["dX"][others], want["dX"][others])
    for k in ("dA", "dB"):
        assert torch.equal(got[k][keep], want[k][keep]), k
