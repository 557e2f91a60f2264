"""What a workspace holds before a call does not reach the layer's results: every output from a
workspace of NaN (all bytes 0xFF) equals, bit for bit, the one from a workspace of zeros.  Ranks
that are no multiple of 16 leave rows of the packed adapter operands that nothing writes, and the
last of a slice's tokens end inside a stage."""

import pytest
import torch

import sparse_rank_adapter_amd as sra

pytestmark = pytest.mark.gpu


def both(f, nbytes, dev):
    outs = []
    for fill in (0, 255):
        outs.append(f(torch.full((max(nbytes, 1),), fill, dtype=torch.uint8, device=dev)))
    torch.cuda.synchronize()
    return outs


def same(a, b, name):
    assert not torch.isnan(b.float()).any(), name
    assert torch.equal(a, b), name


@pytest.mark.parametrize("streaming", [False, True])
@pytest.mark.parametrize("r", [1, 4, 8, 15, 16, 20, 40, 72, 100, 144])
@pytest.mark.parametrize("T", [1, 9, 70, 130, 300])
def test_layer(gpu, T, r, streaming):
    K, N = 384, 256
    g = torch.Generator().manual_seed(1000 * T + r)

    def draw(*shape):
        return torch.randn(*shape, generator=g).bfloat16().to(gpu)
    S = sra.compress(draw(N, K))
    P = sra.double_prune(S)
    if streaming:
        S, P = sra.nm_tile(S), sra.nm_tile(P)
    X, dY, A, B = draw(T, K), draw(T, N), draw(r, K), draw(N, r)
    a, b = both(lambda ws: sra.sparse_lora_fwd(S, X, A, B, ws=ws), sra.fwd_workspace(S, T, r), gpu)
    same(a[0], b[0], "Y")
    same(a[1], b[1], "U")
    U = b[1]
    nb = sra.bwd_workspace(P, T, r)
    a, b = both(lambda ws: sra.sparse_lora_bwd(P, dY, X, U, A, B, ws=ws, want_du=True), nb, gpu)
    for k in a:
        same(a[k], b[k], k)
    a, b = both(lambda ws: sra.sparse_lora_bwd(P, dY, X, U, A, B, ws=ws, dx=False, db=False), nb, gpu)
    same(a["dA"], b["dA"], "dA alone")


def test_infinite_gradient_keeps_to_its_row(gpu):
    """An overflow in one row of dU (dY B) reaches that row of dA alone."""
    T, K, N, r = 9, 384, 256, 16
    g = torch.Generator().manual_seed(5)
    P = sra.double_prune(sra.compress(torch.randn(N, K, generator=g).bfloat16().to(gpu)))
    X, dY = (torch.randn(T, c, generator=g).bfloat16().to(gpu) for c in (K, N))
    A, B = torch.randn(r, K, generator=g).bfloat16().to(gpu), torch.randn(N, r, generator=g).bfloat16().to(gpu)
    U = torch.randn(T, r, generator=g).to(gpu)
    want = sra.sparse_lora_bwd(P, dY, X, U, A, B, dx=False, db=False)["dA"]
    B[:, 7] = float("inf")
    got = sra.sparse_lora_bwd(P, dY, X, U, A, B, dx=False, db=False)["dA"]
    rows = [j for j in range(r) if j != 7]
    assert torch.equal(got[rows], want[rows])
    assert not torch.isfinite(got[7]).any()
