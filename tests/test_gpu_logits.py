"""adjust_logits against a 64-bit reference, word by word: histories of every length, counted in LDS
and through the table, masks that leave nothing, and tokens that are not words."""
import math

import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests import act_ref as ref

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def expected(x, tokens, starts, prompts, rep, pres, freq, bias, allowed):
    """(value, bound) in 64 bits."""
    V, T = x.shape
    y = x.double().clone()
    off = torch.zeros_like(y)
    for t in range(T):
        if tokens is not None:
            own = tokens[starts[t]:starts[t + 1]]
            skip = 0 if prompts is None else int(prompts[t])
            fits = lambda a: a[(a >= 0) & (a < V)]
            seen = torch.bincount(fits(own), minlength=V)
            later = torch.bincount(fits(own[skip:]), minlength=V)
            if rep is not None:
                r = rep[t].double()
                y[:, t] = torch.where(seen > 0, torch.where(y[:, t] > 0, y[:, t] / r, y[:, t] * r), y[:, t])
            size = y[:, t].abs()
            if pres is not None:
                y[:, t] -= pres[t].double() * (later > 0)
                size = size + pres[t].double().abs() * (later > 0)
            if freq is not None:
                y[:, t] -= freq[t].double() * later
                size = size + freq[t].double().abs() * later
            off[:, t] = 4 * ref.F32 * size
        if bias is not None:
            b = (bias if bias.dim() == 1 else bias[:, t]).double()
            y[:, t] += b
            off[:, t] += 2 * ref.F32 * (y[:, t].abs() + b.abs())
        if allowed is not None:
            bit = (allowed[t].long().repeat_interleave(32)[:V] >> (torch.arange(V) % 32)) & 1
            y[:, t] = torch.where(bit > 0, y[:, t], torch.full_like(y[:, t], -math.inf))
    fine = torch.where(torch.isfinite(y), y, torch.zeros_like(y))
    return y, (off + ref.rounding(fine, x.dtype)) * (1 + 2 * ref.HALF[x.dtype])


def history(V, T, longest, seed, spread=None):
    gen = torch.Generator().manual_seed(seed)
    lengths = torch.randint(0, longest + 1, (T,), generator=gen)
    starts = torch.nn.functional.pad(lengths.cumsum(0), (1, 0))
    tokens = torch.randint(-2, (spread or V) + 2, (int(starts[-1]) + 5,), generator=gen)
    prompts = (torch.rand(T, generator=gen) * 1.5 * lengths).long()  # some past the column's end
    return tokens, starts, prompts


def run(V, T, dtype, longest, parts, bias=None, mask=False, seed=0, in_place=False, spread=None):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(V, T, generator=gen) * 4).to(DT[dtype])
    tokens = starts = prompts = None
    if longest is not None:
        tokens, starts, prompts = history(V, T, longest, seed + 1, spread)
        if "prompts" not in parts:
            prompts = None
    draw = lambda name, a, b: (torch.rand(T, generator=gen) * (b - a) + a) if name in parts else None
    rep, pres, freq = draw("rep", 0.7, 1.6), draw("pres", -1, 1), draw("freq", -0.5, 0.5)
    b = None if bias is None else torch.randn((V,) if bias == "shared" else (V, T), generator=gen)
    allowed = None
    if mask:
        allowed = torch.randint(-2 ** 31, 2 ** 31, (T, -(-V // 32)), generator=gen).int()
        allowed[0] = 0
    cuda = lambda t: None if t is None else t.cuda()
    dev = x.cuda()
    got = nm.adjust_logits(dev, cuda(tokens), cuda(starts), cuda(prompts), cuda(rep), cuda(pres),
                           cuda(freq), cuda(b), cuda(allowed), out=dev if in_place else None)
    if in_place:
        assert got is dev
    else:
        assert torch.equal(dev, x.cuda())
    ref.check(got, *expected(x, tokens, starts, prompts, rep, pres, freq, b, allowed), "logits")


ALL = ("rep", "pres", "freq", "prompts")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V,T", [(1, 1), (31, 2), (33, 3), (1000, 1), (8191, 1), (8193, 1), (3001, 5),
                                 (700, 16), (513, 17), (257, 64), (300, 33), (40, 100), (20011, 20)])
def test_sizes(V, T, dtype):
    run(V, T, dtype, 50, ALL, "shared", True)


@pytest.mark.parametrize("parts", [(), ("rep",), ("pres",), ("freq",), ("rep", "prompts"), ALL,
                                   ("rep", "pres", "freq")])
@pytest.mark.parametrize("bias,mask", [(None, False), ("each", True), ("shared", False)])
def test_parts(parts, bias, mask):
    run(500, 9, "fp32", 60, parts, bias, mask)


@pytest.mark.parametrize("T", [7, 40])
@pytest.mark.parametrize("bias,mask", [(None, False), ("each", False), (None, True)])
def test_without_tokens(bias, mask, T):
    run(2000, T, "bf16", None, (), bias, mask)


@pytest.mark.parametrize("longest", [0, 1, 5000])
def test_lengths(longest):
    run(4000, 6, "fp32", longest, ALL)


def test_repeated_words():
    run(3000, 5, "fp32", 4000, ALL, spread=7)


@pytest.mark.parametrize("T,count", [(1, 3_000_000), (40, 700_000)])
def test_long_histories_through_the_table(T, count):
    V = 20000
    assert nm.lib().nm_adjust_logits_workspace_bytes(V, T, count) == V * T * 4
    gen = torch.Generator().manual_seed(8)
    tokens = torch.randint(-1, V + 1, (count,), generator=gen)
    cuts = torch.sort(torch.randint(0, count, (T - 1,), generator=gen)).values
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([count])])
    prompts = torch.randint(0, count // T, (T,), generator=gen)
    x = torch.randn(V, T, generator=gen)
    rep, pres, freq = torch.rand(T, generator=gen) + 1, torch.rand(T, generator=gen), \
        torch.rand(T, generator=gen) * 0.01
    want = expected(x, tokens, starts, prompts, rep, pres, freq, None, None)
    args = [t.cuda() for t in (x, tokens, starts, prompts, rep, pres, freq)]
    first = nm.adjust_logits(*args)
    ref.check(first, *want, "logits")
    assert torch.equal(nm.adjust_logits(*args), first)


def test_in_place():
    run(5000, 12, "fp16", 100, ALL, "each", True, in_place=True)


def test_infinite_logits():
    V, T = 200, 2
    x = torch.randn(V, T)
    x[3], x[4], x[5] = math.inf, -math.inf, math.nan
    tokens = torch.tensor([3, 4, 5, 3, 3, 4])
    starts = torch.tensor([0, 3, 6])
    rep, pres = torch.tensor([1.5, 2.0]), torch.tensor([0.5, 0.5])
    allowed = torch.full((T, 7), -1, dtype=torch.int32)
    allowed[0, 0] = ~(1 << 5)  # the NaN is not allowed in the first column
    got = nm.adjust_logits(x.cuda(), tokens.cuda(), starts.cuda(), repetition=rep.cuda(),
                           presence=pres.cuda(), allowed=allowed.cuda()).cpu()
    assert got[3].tolist() == [math.inf] * 2 and got[4].tolist() == [-math.inf] * 2
    assert got[5, 0] == -math.inf and got[5, 1].isnan()
    assert bool(got[6:].isfinite().all())


def test_starts_that_point_outside_are_held():
    x = torch.randn(100, 3)
    tokens = torch.arange(10)
    starts = torch.tensor([-5, 4, 2, 1000])  # the second column is empty, the third ends with the tokens
    rep = torch.full((3,), 2.0)
    got = nm.adjust_logits(x.cuda(), tokens.cuda(), starts.cuda(), repetition=rep.cuda())
    held = torch.tensor([0, 4, 4, 10])
    want = x.double().clone()
    for t, (a, b) in enumerate(((0, 4), (4, 2), (2, 10))):
        for v in range(a, b):
            want[v, t] = want[v, t] / 2 if want[v, t] > 0 else want[v, t] * 2
    assert held.numel() == 4
    ref.check(got, want, ref.rounding(want, torch.float32), "logits")


def test_views_that_start_anywhere():
    x = torch.randn(300, 2).cuda()
    tokens = torch.randint(0, 300, (41,)).cuda()
    starts = torch.tensor([9, 0, 13, 40]).cuda()
    a = nm.adjust_logits(x, tokens[1:], starts[1:], repetition=torch.ones(3).cuda()[1:] * 2)
    b = nm.adjust_logits(x, tokens[1:].clone(), starts[1:].clone(), repetition=torch.full((2,), 2.0).cuda())
    assert torch.equal(a, b)


def test_refusals():
    x = torch.randn(64, 2).cuda()
    tokens = torch.zeros(3, dtype=torch.int64).cuda()
    starts = torch.tensor([0, 1, 3]).cuda()
    for bad in (dict(tokens=tokens), dict(starts=starts), dict(tokens=tokens.int(), starts=starts),
                dict(tokens=tokens, starts=starts[:2]), dict(bias=torch.zeros(65).cuda()),
                dict(allowed=torch.zeros(2, 3, dtype=torch.int32).cuda()),
                dict(repetition=torch.ones(3).cuda()), dict(out=torch.zeros(64, 3).cuda())):
        with pytest.raises(ValueError):
            nm.adjust_logits(x, **bad)
    with pytest.raises(nm.NMError):
        nm.adjust_logits(x, bias=x, out=x)
