"""Layer norm of rows with no columns checks the outputs it writes (no GPU, no launch)."""
import pytest

from sparse_rank_adapter_amd import _abi
from sparse_rank_adapter_amd._abi import SRA_BF16, SRA_ERR_INVALID_ARG, SRA_OK

FAKE = 1 << 20


@pytest.mark.parametrize("mean,rstd,code", [(FAKE + 2, None, SRA_ERR_INVALID_ARG), (None, FAKE + 8, SRA_ERR_INVALID_ARG),
                                            (None, None, SRA_OK)])
def test_outputs(mean, rstd, code):
    assert _abi.load().sra_layer_norm_fwd(None, None, None, 1e-5, SRA_BF16, 3, 0, None, mean, rstd, None, None, None) == code
