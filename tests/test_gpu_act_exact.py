"""int8 products of spmm_act at rows so long that fp32 alone could not hold their sums: bit for bit the whole
number, rounded once.  (test_more_limits.py holds the rule to the kernel that adds parts of them in fp32.)"""
import pytest
import torch

import masking_sparse_gemm_amd as nm

pytestmark = pytest.mark.gpu

SIZES = [(33, 2 ** 17 - 64, 1), (33, 2 ** 17 - 64, 20), (20, 2 ** 17 - 24, 20), (20, 2 ** 17 - 24, 1)]


def numbers(kind, *shape, seed):
    gen = torch.Generator().manual_seed(seed)
    if kind == "large":   # every product positive, odd ones among them
        return torch.randint(100, 128, shape, generator=gen).to(torch.int8)
    if kind == "least":   # -128, but for a few
        return torch.where(torch.rand(shape, generator=gen) < 0.01, 127, -128).to(torch.int8)
    return torch.randint(-128, 128, shape, generator=gen).to(torch.int8)


@pytest.mark.parametrize("R,K,T", SIZES)
@pytest.mark.parametrize("n,m", [(2, 4), (1, 2), (1, 4), (4, 8)])
@pytest.mark.parametrize("kind", ["large", "least", "any"])
def test_sums_are_whole_numbers(R, K, T, n, m, kind):
    w, x = numbers(kind, R, K, seed=1), numbers(kind, K, T, seed=2)
    values, meta = nm.compress(w.cuda(), n, m)
    dense = nm.decompress(values, meta, n, m, K, rows=R).cpu()
    want = dense.double() @ x.double()   # below 2^31: exact
    # what one of eight waves adds up, steps of 64 in turn: past what fp32 holds
    steps = torch.nn.functional.pad(dense.double() * x.double()[:, 0], (0, -K % 64)).view(R, -1, 64).sum(2)
    wave = steps[:, ::8].sum(1)
    if kind == "large":
        assert bool((wave > 2 ** 24).all()) and bool((wave.float().double() != wave).any())
    got = nm.spmm_act(values, meta, x.cuda(), n, m, out_dtype=torch.float32)
    assert torch.equal(got.cpu(), want.long().float())
