"""Layer norm of rows with no columns: every output is written."""
import pytest
import torch

import sparse_rank_adapter_amd as sra

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [0, 1, 300])
def test_no_columns(gpu, T, dtype):
    X, w = torch.zeros(T, 0, dtype=dtype, device=gpu), torch.zeros(0, dtype=dtype, device=gpu)
    for _ in range(2):  # the second call's buffers may be the first's, changed since
        Y, mean, rstd, c = sra.layer_norm_fwd(X, w, w, ckpt=True)
        assert Y.shape == (T, 0) and c.codes.shape == (T, 0) and c.exps.shape == (T, 0)
        assert bool(torch.isnan(mean).all()) and bool(torch.isnan(rstd).all())  # 0 / 0
        mean.fill_(7.0)
        rstd.fill_(7.0)
        del mean, rstd
    one = torch.ones(T, device=gpu)
    dX, dg, db = sra.layer_norm_bwd(X, X, w, one, one)
    assert dX.shape == (T, 0) and dg.shape == (0,) and db.shape == (0,)
