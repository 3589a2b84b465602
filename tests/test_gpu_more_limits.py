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


@pytest.mark.parametrize("V,T,count", [(2 ** 30, 17, 0), (2 ** 30 - 999, 16, 0), (2 ** 31 - 1, 16, 40)])
def test_logits_of_many_words(V, T, count):
    from tests.test_gpu_logits import expected

    period = 8192
    base = randn(period, T, seed=4)
    x = base.cuda().repeat(-(-V // period), 1)[:V]
    if count == 0:
        shared = torch.randn(period, generator=torch.Generator().manual_seed(5))
        nm.adjust_logits(x, bias=shared.cuda().repeat(-(-V // period))[:V].contiguous(), out=x)
        want = expected(base, None, None, None, None, None, None, shared, None)
    else:
        # words of every part of the vocabulary, at their places modulo the period
        gen = torch.Generator().manual_seed(6)
        tokens = torch.randint(0, V, (count * T,), generator=gen)
        tokens[0], tokens[count] = V - 1, 2 ** 30
        starts = torch.arange(T + 1) * count
        rep = torch.rand(T, generator=gen) + 1
        nm.adjust_logits(x, tokens.cuda(), starts.cuda(), repetition=rep.cuda(), out=x)
        col = torch.arange(T).repeat_interleave(count)
        before = base[tokens % period, col].double()
        after = torch.where(before > 0, before / rep[col].double(), before * rep[col].double())
        got = x[tokens.cuda(), col.cuda()]
        ref.check(got, after, 4 * ref.F32 * after.abs() + ref.rounding(after, BF) * (1 + 2.0 ** -7), "words")
        x[tokens.cuda(), col.cuda()] = base[tokens % period, col].cuda()
        want = expected(base, None, None, None, None, None, None, None, None)
    ref.check(x[:period], *want, "logits")
    first = x[:period].clone()
    for v in range(0, V, 2 ** 28):
        part = x[v:v + 2 ** 28]
        whole = part.shape[0] // period * period
        assert bool((part[:whole].view(-1, period, T) == first).all())
        assert torch.equal(part[whole:], first[:part.shape[0] - whole])
