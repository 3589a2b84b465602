"""The orthogonalised update where eps holds it back: updates far smaller than eps, whose first
X = G / (|G| + eps) is tiny.

The steps multiply a tiny X by 3.4445 each, its relative errors with it, so the bounds of
test_gpu_orth hold; for twelve steps, in which a tiny X grows to singular values near 1, see
BOUND12.
"""
import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests.test_gpu_orth import BOUND, off, plain, update

pytestmark = pytest.mark.gpu

# A CPU model of the fp32 form's roundings (two fp16 parts, fp32 sums) over 8 to 20 steps from an |X|
# of 1e-8 to 1e-3 gives 2e-7 to 1e-6 over sizes and seeds; the bound of five steps is kept.
BOUND12 = BOUND[torch.float32]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nm.lib()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("R,K", [(64, 96), (200, 130)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("factor", [1e-9, 1e-12, 1e-15, 1e-19, 1e-24])
def test_updates_far_below_eps(R, K, dtype, factor):
    G = (update(R, K, torch.float64) * factor).to(dtype)
    for steps in (1, 5):
        got = nm.orthogonalize(G.cuda(), steps=steps)
        assert off(got, plain(G, steps)) <= BOUND[dtype]


def test_fp16_update_far_below_eps():
    """eps far above the update; the results are fp16's normal numbers."""
    G = (update(64, 96, torch.float64) * 1e6).to(torch.float16)   # |G| about 8e4
    got = nm.orthogonalize(G.cuda(), eps=1e8)
    assert off(got, plain(G, eps=1e8)) <= BOUND[torch.float16]


@pytest.mark.parametrize("eps,steps", [(1e-7, 12), (1e-9, 8), (1e-4, 20)])
def test_grows_to_singular_values_near_one(eps, steps):
    G = (update(64, 96, torch.float64) * 1e-11).to(torch.float32)  # |G| about 8e-13
    got = nm.orthogonalize(G.cuda(), steps=steps, eps=eps)
    assert off(got, plain(G, steps, eps)) <= BOUND12


def test_infinite_eps():
    G = update(64, 96, torch.float32)
    assert (nm.orthogonalize(G.cuda(), eps=float("inf")) == 0).all()
