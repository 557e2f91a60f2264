"""The many-adapter backward's workspace query is enough for every call with its flags (no GPU, no launch).

Each call gets the queried number of bytes at an address that is no multiple of 16.  The library checks the
size before the address, so SRA_ERR_WORKSPACE says that the size was too small and SRA_ERR_INVALID_ARG that it
was accepted; the shapes are such that every call below needs a workspace, so none gets further.
"""
import ctypes
import itertools

import pytest

from sparse_rank_adapter_amd import _abi
from sparse_rank_adapter_amd._abi import (SRA_BF16, SRA_ERR_INVALID_ARG, SRA_FMT_NM, SRA_FMT_NM_TILED, SRA_OK,
                                          SraSparse)

FAKE = 1 << 20
CALLS = [(flags, u, du, ckpt) for flags, u, du, ckpt in itertools.product(range(16), (0, 1), (0, 1), (0, 1))
         if flags & 7 or du]


@pytest.mark.parametrize("T,K,N,r,n", [(64, 128, 4096, 16, 8), (75, 128, 4096, 40, 4), (300, 160, 8192, 64, 3),
                                       (1000, 1024, 8192, 130, 1), (40, 20, 4096, 8, 2), (257, 200, 4096, 200, 5)])
@pytest.mark.parametrize("fmt,nn,mm", [(SRA_FMT_NM, 2, 4), (SRA_FMT_NM, 1, 2), (SRA_FMT_NM_TILED, 2, 4), (SRA_FMT_NM, 2, 8)])
def test_query_is_enough(T, K, N, r, n, fmt, nn, mm):
    lib = _abi.load()
    P = SraSparse(fmt, SRA_BF16, K, N, nn, mm, 0, 0, FAKE, FAKE, None, None)
    size = ctypes.c_size_t()
    for flags, u, du, ckpt in CALLS:
        assert lib.sra_multi_bwd_workspace(ctypes.byref(P), T, n, r, flags, ctypes.byref(size)) == SRA_OK
        got = lib.sra_multi_lora_bwd(ctypes.byref(P), FAKE, None if ckpt else FAKE, FAKE if ckpt else None,
                                     FAKE if ckpt else None, T, FAKE if u else None, FAKE, FAKE, FAKE, n, r, flags, FAKE,
                                     FAKE, FAKE, FAKE if du else None, FAKE + 1, size.value, None)
        assert got == SRA_ERR_INVALID_ARG and b"aligned" in lib.sra_last_error(), (flags, u, du, ckpt, lib.sra_last_error())
