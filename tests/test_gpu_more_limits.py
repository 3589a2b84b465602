"""Calls of the epilogue and logits operators on both sides of the sizes where a launch's work-items would
pass 2^32: every row or word against a period of the input, which is checked against the 64-bit form."""
import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests import act_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def empty():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF)


@pytest.mark.parametrize("R,K,T", [(2 ** 27 - 16, 4, 1), (2 ** 27, 4, 1), (2 ** 28 + 5, 4, 2), (2 ** 27, 64, 1),
                                   (2 ** 27 - 31, 64, 1)])
def test_product_of_many_rows(R, K, T):
    period = 4096  # whole tiles of any kernel
    values, meta = nm.compress(randn(period, K, seed=1).cuda(), 2, 4)
    W = nm.decompress(values, meta, 2, 4, K).cpu().double()
    X, b = randn(K, T, seed=2), torch.randn(period, generator=torch.Generator().manual_seed(3))
    n = R // period + 1
    many = lambda t: t.repeat(n, *[1] * (t.dim() - 1))[:R].contiguous()
    Y = nm.spmm_act(many(values), many(meta), X.cuda(), bias=many(b.cuda()), act="silu")
    x = X.double()
    off = ref.sum_bound(K // 2, W.abs() @ x.abs())
    wy, by, _, _ = ref.epilogue(W @ x, off, b, "silu", None, BF)
    ref.check(Y[:period], wy, by, "Y")
    whole = R // period * period
    assert bool((Y[:whole].view(-1, period, T) == Y[:period]).all())
    assert torch.equal(Y[whole:], Y[:R - whole])
