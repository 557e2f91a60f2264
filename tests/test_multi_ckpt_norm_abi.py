"""Host-side refusals of the many-adapter, checkpoint and layer norm calls (no GPU, no launch).

Every call below fails validation or is a pure size query; pointers are fake and never read.
"""
import ctypes
import itertools

import pytest
import torch

from sparse_rank_adapter_amd import _abi, api
from sparse_rank_adapter_amd._abi import (SRA_BF16, SRA_ERR_INVALID_ARG, SRA_ERR_UNSUPPORTED, SRA_ERR_WORKSPACE,
                                          SRA_F32, SRA_FMT_CSR, SRA_FMT_ELL, SRA_FMT_NM, SRA_FMT_NM_TILED, SRA_OK,
                                          SraSparse)
from sparse_rank_adapter_amd.api import Ckpt8, SparseMatrix

FAKE = 1 << 20
ALL = 7


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def nm(rows=64, cols=128, dtype=SRA_BF16, fmt=SRA_FMT_NM, n=2, m=4):
    d = SraSparse()
    d.format, d.dtype, d.rows, d.cols, d.n, d.m = fmt, dtype, rows, cols, n, m
    d.values, d.meta = FAKE, FAKE
    return d


def fwd(lib, d=None, X=FAKE, T=8, A=FAKE, B=FAKE, ids=FAKE, n=4, r=8, Y=FAKE, U=FAKE, ws=FAKE, wsb=1 << 40):
    return lib.sra_multi_lora_fwd(ctypes.byref(d if d is not None else nm()), X, T, A, B, ids, n, r, Y, U, ws, wsb, None)


def bwd(lib, d=None, dY=FAKE, X=FAKE, codes=None, exps=None, T=8, U=FAKE, A=FAKE, B=FAKE, ids=FAKE, n=4, r=8, flags=ALL,
        dX=FAKE, dA=FAKE, dB=FAKE, dU=None, ws=FAKE, wsb=1 << 40):
    return lib.sra_multi_lora_bwd(ctypes.byref(d if d is not None else nm()), dY, X, codes, exps, T, U, A, B, ids, n, r,
                                  flags, dX, dA, dB, dU, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), SRA_ERR_INVALID_ARG), (dict(A=None), SRA_ERR_INVALID_ARG), (dict(B=None), SRA_ERR_INVALID_ARG),
    (dict(ids=None), SRA_ERR_INVALID_ARG), (dict(ids=FAKE + 2), SRA_ERR_INVALID_ARG), (dict(Y=None), SRA_ERR_INVALID_ARG),
    (dict(X=FAKE + 8), SRA_ERR_INVALID_ARG), (dict(U=FAKE + 4), SRA_ERR_INVALID_ARG), (dict(T=-1), SRA_ERR_INVALID_ARG),
    (dict(T=1 << 26), SRA_ERR_UNSUPPORTED), (dict(r=0), SRA_ERR_UNSUPPORTED), (dict(r=257), SRA_ERR_UNSUPPORTED),
    (dict(n=0), SRA_ERR_INVALID_ARG), (dict(n=1024), SRA_ERR_UNSUPPORTED), (dict(U=None, ws=None), SRA_ERR_WORKSPACE),
    (dict(U=None, wsb=16), SRA_ERR_WORKSPACE), (dict(U=None, ws=FAKE + 1), SRA_ERR_INVALID_ARG),
    (dict(d=nm(dtype=SRA_F32)), SRA_ERR_UNSUPPORTED), (dict(d=nm(cols=48)), SRA_ERR_UNSUPPORTED),
    (dict(d=nm(cols=0)), SRA_ERR_UNSUPPORTED), (dict(d=nm(cols=160, fmt=SRA_FMT_NM_TILED), T=17), SRA_ERR_UNSUPPORTED),
    (dict(d=nm(rows=1 << 23), r=256), SRA_ERR_UNSUPPORTED), (dict(d=nm(n=1, m=4)), SRA_ERR_UNSUPPORTED),
])
def test_forward_refusals(lib, kw, code):
    assert fwd(lib, **kw) == code
    assert lib.sra_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(dY=None), SRA_ERR_INVALID_ARG), (dict(X=None), SRA_ERR_INVALID_ARG), (dict(A=None), SRA_ERR_INVALID_ARG),
    (dict(B=None), SRA_ERR_INVALID_ARG), (dict(ids=None), SRA_ERR_INVALID_ARG), (dict(dX=None), SRA_ERR_INVALID_ARG),
    (dict(dA=None), SRA_ERR_INVALID_ARG), (dict(dB=None), SRA_ERR_INVALID_ARG), (dict(flags=16), SRA_ERR_INVALID_ARG),
    (dict(codes=FAKE), SRA_ERR_INVALID_ARG), (dict(codes=FAKE, exps=FAKE), SRA_ERR_INVALID_ARG),  # X twice
    (dict(X=None, codes=FAKE), SRA_ERR_INVALID_ARG), (dict(X=None, codes=FAKE + 1, exps=FAKE), SRA_ERR_INVALID_ARG),
    (dict(U=FAKE + 4), SRA_ERR_INVALID_ARG), (dict(dU=FAKE + 4), SRA_ERR_INVALID_ARG), (dict(wsb=64), SRA_ERR_WORKSPACE),
    (dict(X=None, U=None, flags=4), SRA_ERR_INVALID_ARG), (dict(d=nm(rows=0)), SRA_ERR_UNSUPPORTED),
    (dict(r=300), SRA_ERR_UNSUPPORTED), (dict(n=-1), SRA_ERR_INVALID_ARG), (dict(T=1 << 30), SRA_ERR_UNSUPPORTED),
])
def test_backward_refusals(lib, kw, code):
    assert bwd(lib, **kw) == code
    assert lib.sra_last_error()


@pytest.mark.parametrize("fmt", [SRA_FMT_ELL, SRA_FMT_CSR])
def test_other_formats_are_refused(lib, fmt):
    d = nm(fmt=fmt)
    d.k, d.nnz, d.index, d.row_ptr = 8, 64 * 8, FAKE, FAKE
    assert fwd(lib, d=d) == SRA_ERR_UNSUPPORTED
    assert bwd(lib, d=d) == SRA_ERR_UNSUPPORTED


def test_workspace_sizes_over_the_range(lib):
    """Every size query of the range answers (no division by an empty shape)."""
    out = ctypes.c_size_t()
    for rows, cols, n, r in itertools.product((32, 4096), (32, 96, 1024), (1, 7, 1023), (1, 16, 40, 64, 130, 256)):
        for T in (0, 1, 16, 17, 255, 256, 4099):
            d = nm(rows, cols)
            assert lib.sra_multi_fwd_workspace(ctypes.byref(d), T, n, r, ctypes.byref(out)) == SRA_OK
            if T == 0:
                assert out.value == 0
            for flags in range(16):
                assert lib.sra_multi_bwd_workspace(ctypes.byref(d), T, n, r, flags, ctypes.byref(out)) == SRA_OK
    for fmt, nn, mm in ((SRA_FMT_NM, 1, 2), (SRA_FMT_NM, 2, 8), (SRA_FMT_NM_TILED, 2, 4), (SRA_FMT_NM_TILED, 2, 8)):
        for T in (0, 3, 100):
            d = nm(128, 256, fmt=fmt, n=nn, m=mm)
            assert lib.sra_multi_fwd_workspace(ctypes.byref(d), T, 3, 64, ctypes.byref(out)) == SRA_OK
            assert lib.sra_multi_bwd_workspace(ctypes.byref(d), T, 3, 64, 7, ctypes.byref(out)) == SRA_OK
    assert lib.sra_multi_fwd_workspace(ctypes.byref(nm()), 4, 2, 8, None) == SRA_ERR_INVALID_ARG
    assert lib.sra_multi_bwd_workspace(ctypes.byref(nm()), 4, 2, 8, 7, None) == SRA_ERR_INVALID_ARG


@pytest.mark.parametrize("args,code", [
    ((None, SRA_BF16, 4, 64, FAKE, FAKE), SRA_ERR_INVALID_ARG), ((FAKE, SRA_BF16, 4, 64, None, FAKE), SRA_ERR_INVALID_ARG),
    ((FAKE, SRA_BF16, 4, 64, FAKE, None), SRA_ERR_INVALID_ARG), ((FAKE, 7, 4, 64, FAKE, FAKE), SRA_ERR_INVALID_ARG),
    ((FAKE, SRA_BF16, -1, 64, FAKE, FAKE), SRA_ERR_INVALID_ARG), ((FAKE + 2, SRA_BF16, 4, 64, FAKE, FAKE), SRA_ERR_INVALID_ARG),
])
def test_checkpoint_refusals(lib, args, code):
    assert lib.sra_ckpt_encode(*args, None) == code
    X, dt, T, K, c, e = args
    assert lib.sra_ckpt_decode(c, e, T, K, dt, X, None) == code


def test_masked_weight_grad_ckpt_refusals(lib):
    out = ctypes.c_size_t()
    call = lambda d, row=FAKE, c=FAKE, e=FAKE, T=8, o=FAKE, ws=FAKE, wsb=1 << 40: lib.sra_masked_weight_grad_ckpt(
        ctypes.byref(d), row, c, e, T, o, ws, wsb, None)
    assert call(nm(), row=None) == SRA_ERR_INVALID_ARG
    assert call(nm(), c=None) == SRA_ERR_INVALID_ARG
    assert call(nm(), e=None) == SRA_ERR_INVALID_ARG
    assert call(nm(), o=None) == SRA_ERR_INVALID_ARG
    assert call(nm(), ws=None) == SRA_ERR_WORKSPACE
    assert call(nm(), wsb=100) == SRA_ERR_WORKSPACE
    assert call(nm(rows=60)) == SRA_ERR_UNSUPPORTED
    assert call(nm(dtype=SRA_F32)) == SRA_ERR_UNSUPPORTED
    assert call(nm(), T=1 << 30) == SRA_ERR_UNSUPPORTED
    assert lib.sra_masked_weight_grad_ckpt_workspace(ctypes.byref(nm()), 10, ctypes.byref(out)) == SRA_OK
    assert out.value == 10 * 128 * 2


def ln_fwd(lib, X=FAKE, g=FAKE, b=FAKE, eps=1e-5, dt=SRA_BF16, T=4, H=64, Y=FAKE, m=FAKE, r=FAKE, c=None, e=None):
    return lib.sra_layer_norm_fwd(X, g, b, eps, dt, T, H, Y, m, r, c, e, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), SRA_ERR_INVALID_ARG), (dict(g=None), SRA_ERR_INVALID_ARG), (dict(b=None), SRA_ERR_INVALID_ARG),
    (dict(Y=None), SRA_ERR_INVALID_ARG), (dict(m=None), SRA_ERR_INVALID_ARG), (dict(r=None), SRA_ERR_INVALID_ARG),
    (dict(eps=-1.0), SRA_ERR_INVALID_ARG), (dict(eps=float("nan")), SRA_ERR_INVALID_ARG),
    (dict(eps=float("inf")), SRA_ERR_INVALID_ARG), (dict(dt=9), SRA_ERR_INVALID_ARG), (dict(T=-1), SRA_ERR_INVALID_ARG),
    (dict(H=16385), SRA_ERR_UNSUPPORTED), (dict(c=FAKE), SRA_ERR_INVALID_ARG), (dict(e=FAKE), SRA_ERR_INVALID_ARG),
    (dict(c=FAKE + 3, e=FAKE), SRA_ERR_INVALID_ARG), (dict(T=1 << 31), SRA_ERR_UNSUPPORTED),
])
def test_layer_norm_refusals(lib, kw, code):
    assert ln_fwd(lib, **kw) == code


def test_layer_norm_backward_refusals(lib):
    out = ctypes.c_size_t()
    call = lambda ws=FAKE, wsb=1 << 40, dt=SRA_BF16, T=4, H=64, **p: lib.sra_layer_norm_bwd(
        *[p.get(k, FAKE) for k in ("dY", "X", "g", "m", "r")], dt, T, H,
        *[p.get(k, FAKE) for k in ("dX", "dg", "db")], ws, wsb, None)
    for k in ("dY", "X", "g", "m", "r", "dX", "dg", "db"):
        assert call(**{k: None}) == SRA_ERR_INVALID_ARG, k
    assert call(ws=None) == SRA_ERR_WORKSPACE
    assert call(wsb=8) == SRA_ERR_WORKSPACE
    assert call(H=20000) == SRA_ERR_UNSUPPORTED
    assert lib.sra_layer_norm_bwd_workspace(0, 64, ctypes.byref(out)) == SRA_OK and out.value == 0
    assert lib.sra_layer_norm_bwd_workspace(5, 64, None) == SRA_ERR_INVALID_ARG


# ---- the binding, with the device check replaced by a contiguity check and the library's launches refused
T, K, N, R, G = 12, 64, 96, 8, 3
bf = torch.bfloat16
QUERIES = {"sra_nm_meta_words", "sra_nm_tile_bytes", "sra_multi_fwd_workspace", "sra_multi_bwd_workspace",
           "sra_layer_norm_bwd_workspace", "sra_masked_weight_grad_ckpt_workspace", "sra_last_error"}


@pytest.fixture
def binding(monkeypatch):
    real = _abi.load()

    class HostOnly:
        def __getattr__(self, name):
            if name in QUERIES:
                return getattr(real, name)

            def refuse(*a, **k):
                raise AssertionError(f"{name} reached the library despite invalid arguments")
            return refuse

    def dev_cpu(t, name="tensor", device=None):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t
    monkeypatch.setattr(api, "load", lambda: HostOnly())
    monkeypatch.setattr(api, "_dev", dev_cpu)
    return api


def mat(rows, cols, dtype=bf):
    return SparseMatrix(SRA_FMT_NM, dtype, rows, cols, torch.zeros(rows, cols // 2, dtype=dtype),
                        meta=torch.zeros(rows, cols // 32, dtype=torch.int32))


def z(*s, dt=bf):
    return torch.zeros(*s, dtype=dt)


def kept(t=T, k=K):
    return Ckpt8(z(t, k, dt=torch.int8), z(t, -(-k // 32), dt=torch.uint8))


IDS = z(T, dt=torch.int32)
FWD = dict(Ws=None, X=z(T, K), A=z(G, R, K), B=z(G, N, R), ids=IDS)
BWD = dict(P=None, dY=z(T, N), X=z(T, K), U=z(T, R, dt=torch.float32), A=z(G, R, K), B=z(G, N, R), ids=IDS)


@pytest.mark.parametrize("bad", [
    dict(X=z(T, K + 32)), dict(X=z(T, K, dt=torch.float32)), dict(X=z(K, T).t()), dict(X=z(T, K, 1)),
    dict(A=z(G, R, K + 1)), dict(A=z(R, K)), dict(B=z(G, R, N)), dict(B=z(G + 1, N, R)), dict(B=z(G, N, R, dt=torch.float32)),
    dict(ids=z(T + 1, dt=torch.int32)), dict(ids=z(T, dt=torch.int64)), dict(Y=z(T, N + 1)), dict(U=z(T, R))])
def test_binding_forward(binding, bad):
    with pytest.raises((ValueError, TypeError)):
        binding.multi_lora_fwd(**{**FWD, "Ws": mat(N, K), **bad})


@pytest.mark.parametrize("bad", [
    dict(dY=z(T, K)), dict(X=z(T, N)), dict(X=kept(T + 1)), dict(X=Ckpt8(kept().codes, z(T, 3, dt=torch.uint8))),
    dict(X=Ckpt8(z(T, K), kept().exps)), dict(X=None), dict(X=None, U=None, da=False), dict(U=z(T, R + 1, dt=torch.float32)),
    dict(ids=z(T, 1, dt=torch.int32)), dict(out=dict(dA=z(G, R, K))), dict(out=dict(dX=z(T, K, dt=torch.float32))),
    dict(out=dict(dB=z(G, R, N, dt=torch.float32)))])
def test_binding_backward(binding, bad):
    with pytest.raises((ValueError, TypeError)):
        binding.multi_lora_bwd(**{**BWD, "P": mat(K, N), **bad})


def test_binding_checkpoint_and_norm(binding):
    w = z(K)
    st = z(T, dt=torch.float32)
    bad = [lambda: binding.ckpt8_encode(z(T)), lambda: binding.ckpt8_encode(z(T, K, dt=torch.float16)),
           lambda: binding.ckpt8_encode(z(T, K), out=kept(T, K + 32)),
           lambda: binding.ckpt8_encode(z(T, K, dt=torch.float32), out=kept()), lambda: binding.ckpt8_decode(z(T, K)),
           lambda: binding.ckpt8_decode(kept(), out=z(T, K, dt=torch.float32)),
           lambda: binding.ckpt8_decode(Ckpt8(kept().codes, kept().exps, torch.float16)),
           lambda: binding.layer_norm_fwd(z(T, K), z(K + 1), w), lambda: binding.layer_norm_fwd(z(T, K), w, z(K, dt=torch.float32)),
           lambda: binding.layer_norm_fwd(z(T, K), w, w, ckpt=kept(T, K + 1)), lambda: binding.layer_norm_fwd(z(T), w, w),
           lambda: binding.layer_norm_bwd(z(T, N), z(T, K), w, st, st), lambda: binding.layer_norm_bwd(z(T, K), z(T, K), w, z(T), st),
           lambda: binding.masked_weight_grad(mat(N, K), z(T, N), kept(T, K + 32)),
           lambda: binding.masked_weight_grad(mat(N, K), z(T, N), kept(T + 1, K))]
    for call in bad:
        with pytest.raises((ValueError, TypeError)):
            call()
