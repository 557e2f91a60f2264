"""8-bit floating point codes of rows so long that their tiles do not fit one launch (2^32 threads).

The data repeats every 2^20 columns, whole blocks of 128, so the codes do as well and every part is compared for equality
with those of one period."""
import pytest
import torch

import sparse_rank_adapter_amd as sra

pytestmark = pytest.mark.gpu
PERIOD = 1 << 20


def repeating(cols, gpu):
    base = torch.randn(PERIOD, generator=torch.Generator(device=gpu).manual_seed(3), device=gpu).bfloat16()
    X = torch.empty(1, cols, dtype=torch.bfloat16, device=gpu)
    whole = cols // PERIOD * PERIOD
    X[0, :whole].view(-1, PERIOD).copy_(base.expand(whole // PERIOD, -1))
    X[0, whole:] = base[:cols - whole]
    return base, X


def check_periods(long, one, per, tail):
    """`long` holds `per` values a period, as `one` does, and those of one shorter row behind them."""
    long = long.flatten()
    n = long.numel() // per
    step = max(1, (1 << 30) // per)
    for lo in range(0, n, step):
        k = min(step, n - lo)
        assert (long[lo * per:(lo + k) * per].view(k, per) == one.flatten()).all(), lo
    assert torch.equal(long[n * per:], tail.flatten())


@pytest.mark.parametrize("cols", [(1 << 31) + 40, (1 << 31) + 127])
def test_blocks_of_128_rows(gpu, cols):
    base, X = repeating(cols, gpu)
    got = sra.fp8_encode(X, block_rows=128)
    one, tail = (sra.fp8_encode(base[None, :n].contiguous(), block_rows=128) for n in (PERIOD, cols % PERIOD))
    check_periods(got.codes.view(torch.uint8), one.codes.view(torch.uint8), PERIOD, tail.codes.view(torch.uint8))
    check_periods(got.exps, one.exps, PERIOD // 128, tail.exps)


def test_rows_of_pairs_and_back(gpu):
    cols = (1 << 35) + 2
    torch.cuda.empty_cache()  # 103 GB follow
    base, X = repeating(cols, gpu)
    got = sra.fp8_encode(X)
    one, tail = (sra.fp8_encode(base[None, :n].contiguous()) for n in (PERIOD, cols % PERIOD))
    check_periods(got.codes.view(torch.uint8), one.codes.view(torch.uint8), PERIOD, tail.codes.view(torch.uint8))
    check_periods(got.exps, one.exps, PERIOD // 128, tail.exps)
    back = sra.fp8_decode(got, out=X)
    check_periods(back, sra.fp8_decode(one), PERIOD, sra.fp8_decode(tail))
    del X, got, back
    torch.cuda.empty_cache()
