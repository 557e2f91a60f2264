"""Tensors past 2^31 elements and 2^32 bytes: offsets of the 8-bit floating point, root-mean-square norm and Newton-Schulz
calls.  The operands repeat a short one, so a row's results equal, bit for bit, the short call's where the arithmetic of a
row does not depend on how many there are; sums over the repeats are compared with a bound written beside them.
"""
import pytest
import torch

import sparse_rank_adapter_amd as sra
from oracle import orth as oo

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn
U24 = 2.0 ** -24


def rep(x, n):
    return x.repeat(n, *([1] * (x.dim() - 1)))


def all_equal(big, small, name):
    """big is small, repeated along the rows."""
    if big.dtype == E4:
        big, small = big.view(torch.uint8), small.view(torch.uint8)
    n, k = small.shape[0], big.shape[0] // small.shape[0]
    step = max(1, (1 << 28) // small.numel())
    for i in range(0, k, step):
        part = big[i * n:min(k, i + step) * n]
        assert torch.equal(part, rep(small, part.shape[0] // n)), (name, i)


@pytest.mark.parametrize("C", [1000, 1024])
def test_encode_decode(gpu, C):
    n, k = 1153, 2048  # 2.36e6 rows, 2.36e9 elements and more
    g = torch.Generator().manual_seed(C)
    x = torch.randn(n, C, generator=g).bfloat16().to(gpu)
    f = sra.fp8_encode(x)
    F = sra.fp8_encode(rep(x, k))
    all_equal(F.codes, f.codes, "codes")
    all_equal(F.exps, f.exps, "exps")
    all_equal(sra.fp8_decode(F), sra.fp8_decode(f), "decoded")


@pytest.mark.parametrize("block_rows", [1, 128])
def test_transpose(gpu, block_rows):
    n, C, k = 1152, 1000, 2048  # whole blocks of rows, so every repeat has the same scales
    g = torch.Generator().manual_seed(block_rows)
    x = torch.randn(n, C, generator=g).bfloat16().to(gpu)
    f, ft = sra.fp8_encode_pair(x, E4, block_rows)
    F, Ft = sra.fp8_encode_pair(rep(x, k), E4, block_rows)
    all_equal(F.codes, f.codes, "codes")
    all_equal(F.exps, f.exps, "exps")
    for c in (0, 1, C // 2, C - 1):  # the transpose's rows repeat along their length
        assert torch.equal(Ft.codes[c].view(torch.uint8).view(k, n), ft.codes[c].view(torch.uint8).expand(k, n)), c
    assert torch.equal(Ft.exps.view(Ft.exps.shape[0], k, -1), ft.exps[:, None].expand(-1, k, -1))


@pytest.mark.parametrize("M", [3, 40, 300])
def test_matmul_long_weight(gpu, M):
    n, K, k = 1100, 4096, 1024  # b of 4.6e9 bytes
    g = torch.Generator().manual_seed(M)
    a = sra.fp8_encode(torch.randn(M, K, generator=g).bfloat16().to(gpu))
    w = torch.randn(n, K, generator=g).bfloat16().to(gpu)
    b = sra.fp8_encode(w)
    B = sra.Fp8Matrix(rep(b.codes.view(torch.uint8), k).view(E4), rep(b.exps, k), n * k, K)
    want = sra.fp8_matmul(a, b, out_dtype=torch.float32)
    got = sra.fp8_matmul(a, B, out_dtype=torch.float32).view(M, k, n)
    # fp32 sums of the same exact products in another order: at most K roundings of 2^-24 of the sum of magnitudes each
    mag = (sra.fp8_decode(a, torch.float32).abs() @ sra.fp8_decode(b, torch.float32).abs().t())
    for i in (0, 1, k // 2, k - 2, k - 1):
        assert ((got[:, i] - want).abs() <= 2 * K * U24 * mag).all(), i


@pytest.mark.parametrize("N", [24, 700])
def test_matmul_long_activations(gpu, N):
    n, K, k = 1152, 1024, 4096  # a of 4.8e9 bytes; with N = 700 a result of 3.3e9 elements
    g = torch.Generator().manual_seed(N)
    a = sra.fp8_encode(torch.randn(n, K, generator=g).bfloat16().to(gpu))
    b = sra.fp8_encode(torch.randn(N, K, generator=g).bfloat16().to(gpu), E4, 128)
    A = sra.Fp8Matrix(rep(a.codes.view(torch.uint8), k).view(E4), rep(a.exps, k), n * k, K)
    got = sra.fp8_matmul(A, b)
    want = sra.fp8_matmul(a, b).float()
    mag = (sra.fp8_decode(a, torch.float32).abs() @ sra.fp8_decode(b, torch.float32).abs().t())
    # both rounded to bf16 (2^-8 each) from sums that differ as above, with 2^-17 a step of the 8-bit matrix instruction
    tol = 2 * 2.0 ** -8 * want.abs() + 2 * (K // 128) * 2.0 ** -16 * mag
    for i in (0, 1, k // 2, k - 2, k - 1):
        assert ((got[i * n:(i + 1) * n].float() - want).abs() <= tol).all(), i


def test_rms_norm(gpu):
    n, H, k = 1153, 1000, 2048
    g = torch.Generator().manual_seed(0)
    x, r, dy = (torch.randn(n, H, generator=g).bfloat16().to(gpu) for _ in range(3))
    ga = torch.randn(H, generator=g).bfloat16().to(gpu)
    y, h, rs, f = sra.rms_norm_fwd(x, ga, residual=r, fp8=E4)
    X = rep(x, k)
    Y, Hh, RS, F = sra.rms_norm_fwd(X, ga, residual=rep(r, k), fp8=E4, H=X)
    for name, big, small in (("Y", Y, y), ("H", Hh, h), ("codes", F.codes, f.codes), ("exps", F.exps, f.exps), ("rstd", RS, rs)):
        all_equal(big, small, name)
    del Y, F
    dx, dg = sra.rms_norm_bwd(dy, h, ga, rs)
    dX, dG = sra.rms_norm_bwd(rep(dy, k), Hh, ga, RS)
    all_equal(dX, dx, "dX")
    # T / 512 + 512 fp32 additions of terms with a rounding each
    mag = (dy.double() * h.double() * rs.double()[:, None]).abs().sum(0) * k
    want = (dy.double() * h.double() * rs.double()[:, None]).sum(0) * k
    assert ((dG.double() - want).abs() <= (n * k / 512 + 512 + 3) * U24 * mag).all()


@pytest.mark.parametrize("tall", [False, True])
def test_orthogonalize(gpu, tall):
    """A matrix of 2^31 bytes and more (past 32-bit offsets), its columns a short one's repeated: the result is the short
    one's over sqrt(k), and likewise repeated."""
    d, n, k = 8, 1001, 68000
    g = torch.Generator().manual_seed(int(tall))
    G = torch.randn(d, n, generator=g)
    want = oo.orthogonalize(G.double().numpy(), 5, (3.4445, -4.7750, 2.0315), 0.0) / k ** 0.5
    G = G.to(gpu)
    if tall:
        O = sra.orthogonalize(G.t().contiguous().repeat(k, 1), eps=0.0)
        parts = [O[i * n:(i + 1) * n].t() for i in (0, k // 2, k - 1)]
    else:
        O = sra.orthogonalize(G.repeat(1, k), eps=0.0)
        parts = [O[:, i * n:(i + 1) * n] for i in (0, k // 2, k - 1)]
    want = torch.from_numpy(want)
    # one rounding to fp32; the Gram matrix's sums have under 10^4 fp64 additions in a row (1e-12 of it), and five steps
    # make at most 3.4445^5 = 485 of that
    for p in parts:
        assert ((p.double().cpu() - want).abs() <= 4 * U24 * want.abs() + 1e-9 * want.abs().max()).all()
