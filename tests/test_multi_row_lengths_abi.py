"""The many-adapter backward takes weights of any number of rows K: the workspace query makes room for the
copy of X that row lengths need which the gradient kernels' vector loads do not fit (no GPU, no launch)."""
import ctypes

import pytest

from sparse_rank_adapter_amd import _abi
from sparse_rank_adapter_amd._abi import SRA_BF16, SRA_FMT_NM, SRA_OK, SraSparse

FAKE = 1 << 20
DX, DA, DB = 1, 2, 4


def size(rows, r, flags, T=4096, n=8, cols=128):
    d = SraSparse(SRA_FMT_NM, SRA_BF16, rows, cols, 2, 4, 0, 0, FAKE, FAKE, None, None)
    out = ctypes.c_size_t()
    assert _abi.load().sra_multi_bwd_workspace(ctypes.byref(d), T, n, r, flags, ctypes.byref(out)) == SRA_OK
    return out.value


@pytest.mark.parametrize("rows,r", [(1, 16), (4, 16), (7, 40), (20, 16), (20, 40), (24, 40), (100, 40), (1000, 130)])
def test_room_for_whole_rows(rows, r):
    whole = -(-rows // 32) * 32
    # everything else grows with the rows, so the copy [T, whole] in bf16 is what the shorter rows add
    grads = 2 * 8 * r * 32 * 4  # at most: two slices of partials of the up to 31 columns that differ
    assert size(rows, r, DA) - size(whole, r, DA) >= 4096 * whole * 2 - grads - 4096


@pytest.mark.parametrize("rows,r", [(32, 40), (24, 16), (8, 32), (48, 130)])
def test_none_where_the_loads_fit(rows, r):
    assert size(rows, r, DA) <= size(-(-rows // 32) * 32, r, DA)


@pytest.mark.parametrize("rows", [20, 1000])
def test_none_without_da(rows):
    assert size(rows, 16, DX) <= size(-(-rows // 32) * 32, 16, DX)
