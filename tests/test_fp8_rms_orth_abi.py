"""Host-side refusals of the 8-bit floating point, root-mean-square norm and Newton-Schulz calls (no GPU, no launch).

Every call below fails validation or is a pure size query; pointers are fake and never read.
"""
import ctypes
import itertools

import pytest
import torch

from sparse_rank_adapter_amd import _abi, api
from sparse_rank_adapter_amd._abi import (SRA_BF16, SRA_ERR_INVALID_ARG, SRA_ERR_UNSUPPORTED, SRA_ERR_WORKSPACE, SRA_F32,
                                          SRA_OK, SraFp8)

FAKE = 1 << 20
BAD, UNS, WS = SRA_ERR_INVALID_ARG, SRA_ERR_UNSUPPORTED, SRA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def fp8(rows=64, cols=256, kind=0, block_rows=1, codes=FAKE, exps=FAKE):
    return SraFp8(kind, block_rows, rows, cols, codes, exps)


def ref(d):
    return None if d is None else ctypes.byref(d)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), BAD), (dict(X=FAKE + 4), BAD), (dict(R=FAKE + 8), BAD), (dict(gamma=None), BAD), (dict(Hout=None), BAD),
    (dict(Y=None, codes=None, exps=None), BAD), (dict(Y=FAKE + 2), BAD), (dict(rstd=None), BAD), (dict(codes=None), BAD),
    (dict(exps=None), BAD), (dict(codes=FAKE + 1), BAD), (dict(dt=5), BAD), (dict(T=-1), BAD), (dict(H=-1), BAD),
    (dict(H=16385), UNS), (dict(T=1 << 31), UNS), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
])
def test_rms_forward_refusals(lib, kw, code):
    a = dict(X=FAKE, R=FAKE, gamma=FAKE, eps=1e-6, dt=SRA_BF16, T=4, H=64, Hout=FAKE, Y=FAKE, rstd=FAKE, codes=FAKE, exps=FAKE)
    a.update(kw)
    assert lib.sra_rms_norm_fwd(*a.values(), None) == code
    assert lib.sra_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(dY=None), BAD), (dict(H=None), BAD), (dict(gamma=None), BAD), (dict(rstd=None), BAD), (dict(dH=FAKE + 8), BAD),
    (dict(dX=None), BAD), (dict(dgamma=None), BAD), (dict(ws=None), WS), (dict(wsb=4 * 64 * 4 - 1), WS), (dict(ws=FAKE + 4), BAD),
    (dict(dt=2), BAD), (dict(T=-5), BAD), (dict(W=20000), UNS),
])
def test_rms_backward_refusals(lib, kw, code):
    a = dict(dY=FAKE, H=FAKE, gamma=FAKE, rstd=FAKE, dH=FAKE, dt=SRA_F32, T=4, W=64, dX=FAKE, dgamma=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    assert lib.sra_rms_norm_bwd(*a.values(), None) == code
    assert lib.sra_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), BAD), (dict(dt=9), BAD), (dict(out=None, out_t=None), BAD), (dict(out=fp8(64, 255)), BAD),
    (dict(out_t=fp8(64, 256)), BAD), (dict(out=fp8(kind=2)), BAD), (dict(out=fp8(block_rows=64)), BAD), (dict(out=fp8(codes=None)), BAD),
    (dict(out=fp8(exps=None)), BAD), (dict(out=fp8(codes=FAKE + 8)), BAD), (dict(out_t=fp8(256, 64, kind=1)), BAD),
    (dict(out_t=fp8(256, 64, block_rows=128)), BAD), (dict(rows=-1, out=fp8(-1), out_t=None), BAD),
    (dict(rows=1 << 40, out=fp8(1 << 40), out_t=None), UNS),
])
def test_encode_refusals(lib, kw, code):
    a = dict(X=FAKE, dt=SRA_BF16, rows=64, cols=256, out=fp8(), out_t=fp8(256, 64))
    a.update(kw)
    assert lib.sra_quant_encode(a["X"], a["dt"], a["rows"], a["cols"], ref(a["out"]), ref(a["out_t"]), None) == code
    assert lib.sra_last_error()


@pytest.mark.parametrize("F,dt,X,code", [(None, 0, FAKE, BAD), (fp8(), 3, FAKE, BAD), (fp8(), 0, None, BAD), (fp8(), 0, FAKE + 2, BAD),
                                         (fp8(kind=-1), 0, FAKE, BAD), (fp8(block_rows=0), 0, FAKE, BAD)])
def test_decode_refusals(lib, F, dt, X, code):
    assert lib.sra_quant_decode(ref(F), dt, X, None) == code
    assert lib.sra_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), BAD), (dict(b=None), BAD), (dict(b=fp8(64, 128)), BAD), (dict(dt=7), BAD), (dict(out=None), BAD), (dict(out=FAKE + 8), BAD),
    (dict(a=fp8(codes=None)), BAD), (dict(b=fp8(exps=FAKE + 1)), BAD), (dict(a=fp8(1 << 31)), UNS), (dict(b=fp8(1 << 26)), UNS),
    (dict(a=fp8(64, 1 << 23), b=fp8(64, 1 << 23)), UNS), (dict(a=fp8(1 << 20), b=fp8(1 << 20)), UNS),
    (dict(a=fp8(100, 6000), b=fp8(500, 6000), ws=None), WS), (dict(a=fp8(100, 6000), b=fp8(500, 6000), wsb=100), WS),
    (dict(a=fp8(100, 6000), b=fp8(500, 6000), ws=FAKE + 8), BAD),
])
def test_matmul_refusals(lib, kw, code):
    a = dict(a=fp8(), b=fp8(32, 256, block_rows=128), dt=SRA_BF16, out=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    assert lib.sra_quant_matmul(ref(a["a"]), ref(a["b"]), a["dt"], a["out"], a["ws"], a["wsb"], None) == code
    assert lib.sra_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(G=None), BAD), (dict(O=None), BAD), (dict(G=FAKE + 4), BAD), (dict(dt=4), BAD), (dict(n=-1), BAD), (dict(R=-1), BAD),
    (dict(R=257, C=257), UNS), (dict(n=65536), UNS), (dict(C=1 << 31), UNS), (dict(steps=0), BAD), (dict(steps=65), BAD),
    (dict(a=float("inf")), BAD), (dict(b=float("nan")), BAD), (dict(c=-float("inf")), BAD), (dict(eps=-1e-9), BAD),
    (dict(eps=float("inf")), BAD), (dict(ws=None), WS), (dict(wsb=64), WS), (dict(ws=FAKE + 8), BAD),
    (dict(O=FAKE), BAD), (dict(O=FAKE + 16), BAD), (dict(O=FAKE + 2 * 16 * 100 * 4 - 16), BAD),  # overlap
])
def test_orthogonalize_refusals(lib, kw, code):
    a = dict(G=FAKE, dt=SRA_F32, n=2, R=16, C=100, steps=5, a=3.0, b=-4.0, c=2.0, eps=1e-7, O=FAKE << 4, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    assert lib.sra_orthogonalize(*a.values(), None) == code
    assert lib.sra_last_error()


def test_workspace_sizes_over_the_range(lib):
    n = ctypes.c_size_t()
    for T, H in itertools.product((0, 1, 511, 513, 1 << 30), (0, 1, 129, 16384)):
        assert lib.sra_rms_norm_bwd_workspace(T, H, ctypes.byref(n)) == SRA_OK and n.value == min(T, 512) * H * 4
    for M, N, K in itertools.product((0, 1, 16, 65, 300, 5000), (0, 1, 100, 4097), (0, 1, 127, 2048, 1 << 22)):
        assert lib.sra_quant_matmul_workspace(M, N, K, ctypes.byref(n)) == SRA_OK
        assert n.value % (4 * max(1, M * N)) == 0
    for c, R, C in itertools.product((0, 1, 12, 65535), (0, 1, 16, 33, 64, 65, 256), (0, 1, 100, 256, 20480)):
        assert lib.sra_orthogonalize_workspace(c, R, C, ctypes.byref(n)) == SRA_OK
        assert (n.value == 0) == (c == 0 or R == 0 or C == 0)
        assert lib.sra_orthogonalize_workspace(c, C, R, ctypes.byref(n)) == SRA_OK
    assert lib.sra_rms_norm_bwd_workspace(4, 64, None) == BAD
    assert lib.sra_quant_matmul_workspace(4, 64, 64, None) == BAD
    assert lib.sra_orthogonalize_workspace(4, 64, 64, None) == BAD


def test_kernel_classes(lib):
    assert lib.sra_time_next_kernel(16, FAKE, FAKE) == BAD
    for which in range(12, 16):
        assert lib.sra_time_next_kernel(which, FAKE, FAKE) == SRA_OK
    assert lib.sra_time_next_kernel(0, None, None) == SRA_OK


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape).to(dtype)


def matrix(rows=8, cols=200, kind=torch.float8_e4m3fn, block_rows=1, **kw):
    nb = -(-cols // 128)
    F = api.Fp8Matrix(torch.zeros(rows, nb * 128).to(kind), torch.zeros(-(-rows // block_rows), nb, dtype=torch.uint8), rows, cols, block_rows)
    for k, v in kw.items():
        setattr(F, k, v)
    return F


X = cpu(4, 64)
G = cpu(64)


@pytest.mark.parametrize("call,text", [
    (lambda: api.rms_norm_fwd(cpu(4), G), "2-D"), (lambda: api.rms_norm_fwd(cpu(4, 64, dtype=torch.float16), G), "float16"),
    (lambda: api.rms_norm_fwd(X, cpu(4)), "GPU"), (lambda: api.fp8_encode(cpu(3, 4), torch.float16), "GPU|float16"),
    (lambda: api.fp8_decode(X), "Fp8Matrix"), (lambda: api.fp8_matmul(matrix(), X), "GPU|Fp8Matrix"),
    (lambda: api.fp8_matmul(matrix(block_rows=64), matrix()), "block_rows"), (lambda: api.fp8_matmul(matrix(codes=cpu(8, 256)), matrix()), "float8"),
    (lambda: api.fp8_matmul(matrix(codes=torch.zeros(8, 200).to(torch.float8_e4m3fn)), matrix()), "shape"),
    (lambda: api.fp8_matmul(matrix(exps=torch.zeros(8, 1, dtype=torch.uint8)), matrix()), "GPU|shape"),
    (lambda: api.orthogonalize(cpu(4)), "2-D or 3-D"), (lambda: api.orthogonalize(cpu(4, 5, dtype=torch.float64)), "float64"),
    (lambda: api.orthogonalize(cpu(4, 5)), "GPU"),
])
def test_binding_refuses_before_the_library(call, text):
    with pytest.raises((ValueError, TypeError), match=text):
        call()
