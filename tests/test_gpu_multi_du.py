"""The many-adapter backward asked for dU beside any other gradients, or for dU alone."""
import numpy as np
import pytest

import sparse_rank_adapter_amd as sra
from _util import bits
from test_gpu_multi import run

pytestmark = pytest.mark.gpu
KEYS = dict(dx="dX", da="dA", db="dB")


@pytest.mark.parametrize("T,r", [(12, 8), (75, 16), (300, 40)])
def test_du_with_any_gradients(gpu, T, r):
    S, P, X, dY, A, B, di, U, res = run(gpu, T, 128, 96, r, 4, "mixed")
    full = res["bf16"]
    plain = sra.multi_lora_bwd(P, dY, X, U, A, B, di, da=False, db=False, dx_adapter=False)["dX"]
    for bit in range(16):
        want = {k: bool(bit >> i & 1) for i, k in enumerate(KEYS)}
        got = sra.multi_lora_bwd(P, dY, X, U, A, B, di, **want, dx_adapter=not bit & 8, want_du=True)
        assert set(got) == {"dU"} | {KEYS[k] for k in KEYS if want[k]}
        for k, v in got.items():
            ref = plain if k == "dX" and bit & 8 else full[k]
            assert np.array_equal(bits(v), bits(ref)), (bit, k)
