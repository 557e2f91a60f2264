"""Buffers that overlap where a call would read what it has written are refused (no GPU, no launch: pointers are fake)."""
import ctypes

import pytest

from sparse_rank_adapter_amd import _abi
from sparse_rank_adapter_amd._abi import SRA_BF16, SRA_ERR_INVALID_ARG, SRA_F32, SraFp8

A = 1 << 30
T, H = 4, 256
N = T * H * 2  # bytes of a [T, H] tensor in bf16
AT = [A + k * (1 << 20) for k in range(8)]


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def refused(lib, status):
    assert status == SRA_ERR_INVALID_ARG
    assert b"overlap" in lib.sra_last_error()


@pytest.mark.parametrize("kw", [dict(Hout=AT[0] + 16), dict(Hout=AT[1] - 16), dict(Y=AT[0]), dict(Y=AT[1]), dict(Y=AT[2]),
                                dict(Y=AT[2] + N - 16), dict(codes=AT[0]), dict(codes=AT[1] + 512), dict(codes=AT[2]), dict(codes=AT[3])])
def test_rms_forward(lib, kw):
    a = dict(X=AT[0], R=AT[1], gamma=AT[6], eps=1e-6, dt=SRA_BF16, T=T, H=H, Hout=AT[2], Y=AT[3], rstd=AT[7], codes=AT[4], exps=AT[5])
    a.update(kw)
    refused(lib, lib.sra_rms_norm_fwd(*a.values(), None))


@pytest.mark.parametrize("off", [16, -16, N - 16])
@pytest.mark.parametrize("k", [0, 1, 2])
def test_rms_backward(lib, k, off):
    refused(lib, lib.sra_rms_norm_bwd(AT[0], AT[1], AT[5], AT[6], AT[2], SRA_BF16, T, H, AT[k] + off, AT[7], A - (1 << 28), 1 << 20, None))


@pytest.mark.parametrize("c,t", [(AT[0], AT[2]), (AT[1], AT[0] + 2032), (AT[1], AT[1] + 512), (AT[0] + N - 16, None), (None, AT[0] - 16)])
def test_encode(lib, c, t):
    out = SraFp8(0, 1, T, H, c, AT[6]) if c else None
    out_t = SraFp8(0, 1, H, T, t, AT[7]) if t else None
    refused(lib, lib.sra_quant_encode(AT[0], SRA_BF16, T, H, ctypes.byref(out) if out else None, ctypes.byref(out_t) if out_t else None, None))


def test_decode(lib):
    refused(lib, lib.sra_quant_decode(ctypes.byref(SraFp8(0, 1, T, H, AT[1], AT[6])), SRA_F32, AT[1] - T * H * 4 + 16, None))


@pytest.mark.parametrize("o", [AT[0] + 16, AT[1] - 16])
def test_matmul(lib, o):
    a, b = SraFp8(0, 1, T, H, AT[0], AT[6]), SraFp8(0, 1, T, H, AT[1], AT[7])
    refused(lib, lib.sra_quant_matmul(ctypes.byref(a), ctypes.byref(b), SRA_F32, o, None, 0, None))


def test_orthogonalize(lib):
    refused(lib, lib.sra_orthogonalize(AT[0], SRA_BF16, 1, T, H, 5, 3.4, -4.7, 2.0, 1e-7, AT[0] + N - 16, AT[4], 1 << 40, None))
