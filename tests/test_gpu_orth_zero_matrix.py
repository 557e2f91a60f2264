"""A zero matrix stays zero under any eps > 0: the factor 1 / eps is multiplied with itself up to five times, past fp64's range
for the smallest, and zeros times infinity are NaN."""
import pytest
import torch

import sparse_rank_adapter_amd as sra

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [1e-7, 1e-80, 1e-160, 1e-300, 5e-324, 1e300])
@pytest.mark.parametrize("d", [3, 16, 32, 64, 65, 128, 256])
@pytest.mark.parametrize("steps", [1, 2, 5])
def test_zero_matrix(gpu, d, eps, steps):
    G = torch.zeros(3, d, 300, device=gpu)
    G[1].normal_(generator=torch.Generator(device=gpu).manual_seed(d))
    for X in (G, G.transpose(1, 2).contiguous(), G.bfloat16()):
        got = sra.orthogonalize(X, steps=steps, eps=eps)
        assert not got[0].any() and not got[2].any()
        whole = sra.orthogonalize(X[1:2].expand(3, -1, -1).contiguous(), steps=steps, eps=eps)  # a neighbour changes nothing
        assert torch.isfinite(got[1]).all() and torch.equal(got[1], whole[1])


@pytest.mark.parametrize("d", [16, 64, 128])
def test_smallest_values(gpu, d):
    """The smallest nonzero matrix, under an eps far below it: its direction comes back."""
    G = torch.zeros(d, 300, device=gpu)
    G[0, 0] = 2.0 ** -149
    for eps in (1e-60, 1e-300):
        got = sra.orthogonalize(G, steps=1, coeffs=(1.5, -0.5, 0.0), eps=eps)
        want = torch.zeros_like(G)
        want[0, 0] = 1.0  # 1.5 - 0.5 of X = 1
        assert torch.equal(got, want)


@pytest.mark.parametrize("d", [16, 64, 128])
def test_zero_matrix_without_eps(gpu, d):
    """0 / 0: the formula's own NaN."""
    assert torch.isnan(sra.orthogonalize(torch.zeros(d, 300, device=gpu), eps=0.0)).all()
