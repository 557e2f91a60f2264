"""Every output of the root-mean-square norm, 8-bit floating point and Newton-Schulz calls is held against every other
buffer of the call: scales, statistics, weights and workspaces too (no GPU, no launch: pointers are fake)."""
import ctypes

import pytest

from sparse_rank_adapter_amd import _abi
from sparse_rank_adapter_amd._abi import SRA_BF16, SRA_ERR_INVALID_ARG, SRA_F32, SraFp8

A, T, H = 1 << 30, 4, 256
AT = [A + k * (1 << 20) for k in range(12)]


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def refused(lib, status):
    assert status == SRA_ERR_INVALID_ARG
    assert b"overlap" in lib.sra_last_error()


FWD = dict(X=AT[0], R=AT[1], gamma=AT[2], eps=1e-6, dt=SRA_BF16, T=T, H=H, Hout=AT[3], Y=AT[4], rstd=AT[5], codes=AT[6], exps=AT[7])
READ = dict(X=2 * T * H, R=2 * T * H, gamma=2 * H)
WRITE = dict(Hout=2 * T * H, Y=2 * T * H, rstd=4 * T, codes=T * H, exps=T * H // 128)


@pytest.mark.parametrize("out", WRITE)
@pytest.mark.parametrize("other", [*READ, *WRITE])
def test_rms_forward(lib, out, other):
    if out == other:
        return
    size = {**READ, **WRITE}[other]
    for at in (FWD[other], FWD[other] + (size - 1) // 16 * 16):  # its first and its last bytes
        if out == "Hout" and other in ("X", "R") and at == FWD[other]:
            continue  # that one is allowed
        a = dict(FWD)
        a[out] = at
        refused(lib, lib.sra_rms_norm_fwd(*a.values(), None))


BWD = dict(dY=AT[0], Hin=AT[1], gamma=AT[2], rstd=AT[3], dH=AT[4], dt=SRA_BF16, T=T, H=H, dX=AT[5], dgamma=AT[6], ws=AT[7], wsb=1 << 20)
BWD_SIZE = dict(dY=2 * T * H, Hin=2 * T * H, gamma=2 * H, rstd=4 * T, dH=2 * T * H, dX=2 * T * H, dgamma=4 * H, ws=4 * T * H)


@pytest.mark.parametrize("out", ["dX", "dgamma", "ws"])
@pytest.mark.parametrize("other", BWD_SIZE)
def test_rms_backward(lib, out, other):
    if out == other or (out == "dX" and other in ("dY", "Hin", "dH")):
        return
    for at in (BWD[other], BWD[other] + (BWD_SIZE[other] - 1) // 16 * 16):
        a = dict(BWD)
        a[out] = at
        refused(lib, lib.sra_rms_norm_bwd(*a.values(), None))


def test_encode(lib):
    n = dict(x=AT[0], c=AT[1], e=AT[2], ct=AT[3], et=AT[4])
    size = dict(x=2 * T * H, c=T * H, e=T * H // 128, ct=128 * H, et=H)
    for out in ("c", "e", "ct", "et"):
        for other in n:
            if other == out:
                continue
            for at in (n[other], n[other] + (size[other] - 1) // 16 * 16):
                a = dict(n)
                a[out] = at
                f, g = SraFp8(0, 1, T, H, a["c"], a["e"]), SraFp8(0, 1, H, T, a["ct"], a["et"])
                refused(lib, lib.sra_quant_encode(a["x"], SRA_BF16, T, H, ctypes.byref(f), ctypes.byref(g), None))


@pytest.mark.parametrize("block_rows,last", [(1, 32), (128, 0)])
def test_decode(lib, block_rows, last):
    f = SraFp8(0, block_rows, 20, H, AT[0], AT[1])  # 40 exponents, or two
    for at in (AT[1] + last, AT[1] - 20 * H * 4 + 16, AT[0] + 20 * H - 16):
        refused(lib, lib.sra_quant_decode(ctypes.byref(f), SRA_F32, at, None))


def test_matmul(lib):
    M, N, K = 100, 64, 1024
    need = ctypes.c_size_t()
    assert lib.sra_quant_matmul_workspace(M, N, K, ctypes.byref(need)) == 0 and need.value > 0
    at = dict(ac=AT[0], ae=AT[1], bc=AT[2], be=AT[3], out=AT[4], ws=AT[5])
    size = dict(ac=M * K, ae=M * K // 128, bc=N * K, be=K // 128, out=4 * M * N, ws=need.value)
    for w in ("out", "ws"):
        for other in at:
            if other == w:
                continue
            for p in (at[other], at[other] + (size[other] - 1) // 16 * 16):
                x = dict(at)
                x[w] = p
                a, b = SraFp8(0, 1, M, K, x["ac"], x["ae"]), SraFp8(0, 128, N, K, x["bc"], x["be"])
                refused(lib, lib.sra_quant_matmul(ctypes.byref(a), ctypes.byref(b), SRA_F32, x["out"], x["ws"], 1 << 30, None))


def test_orthogonalize(lib):
    call = lambda g, o, ws: lib.sra_orthogonalize(g, SRA_BF16, 1, T, H, 5, 3.4, -4.7, 2.0, 1e-7, o, ws, 1 << 40, None)
    for o, ws in ((AT[0], AT[2]), (AT[1], AT[0]), (AT[1], AT[0] + 2 * T * H - 16), (AT[1], AT[1]), (AT[1], AT[1] + 2 * T * H - 16)):
        refused(lib, call(AT[0], o, ws))
