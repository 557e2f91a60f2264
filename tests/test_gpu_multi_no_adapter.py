"""The many-adapter backward's dX without the adapters needs no ids, A, B, U or X."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_rank_adapter_amd as sra
from sparse_rank_adapter_amd import _abi
from _util import bits, f64
from test_gpu_multi import BF, U24, close, weight

pytestmark = pytest.mark.gpu
DX, NO_ADAPTER = 1, 8


@pytest.mark.parametrize("fmt", [(2, 4), (1, 2), (2, 8)])
@pytest.mark.parametrize("T,K,N", [(4, 64, 128), (40, 96, 1024), (300, 256, 96)])
def test_dx_alone(gpu, T, K, N, fmt):
    g = torch.Generator().manual_seed(T)
    P, Pd = weight(K, N, *fmt, g, gpu)
    dY = torch.randn(T, N, generator=g).bfloat16().to(gpu)
    dX = torch.empty(T, K, dtype=torch.bfloat16, device=gpu)
    lib, d, size = _abi.load(), P.desc(), ctypes.c_size_t()
    assert lib.sra_multi_bwd_workspace(ctypes.byref(d), T, 3, 8, DX | NO_ADAPTER, ctypes.byref(size)) == _abi.SRA_OK
    ws = torch.empty(max(1, size.value), dtype=torch.uint8, device=gpu)
    code = lib.sra_multi_lora_bwd(ctypes.byref(d), dY.data_ptr(), None, None, None, T, None, None, None, None, 3, 8,
                                  DX | NO_ADAPTER, dX.data_ptr(), None, None, None, ws.data_ptr(), size.value,
                                  torch.cuda.current_stream(gpu).cuda_stream)
    assert code == _abi.SRA_OK, lib.sra_last_error()
    want, mag = f64(dY) @ Pd.T, np.abs(f64(dY)) @ np.abs(Pd).T
    close("dX", f64(dX), want, BF * np.abs(want) + (N // 16 + 64) * U24 * mag)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=gpu)
    ids = torch.zeros(T, dtype=torch.int32, device=gpu)
    same = sra.multi_lora_bwd(P, dY, None, None, z(3, 8, K), z(3, N, 8), ids, da=False, db=False, dx_adapter=False)
    assert np.array_equal(bits(dX), bits(same["dX"]))
