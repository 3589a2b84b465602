"""Cross entropy where numbers leave the ordinary range, against plain 64-bit forms.

Where results are infinite or NaN the patterns must be those of the definition in 64 bits.  The
finite ones are held to test_gpu_xent's derivation.
"""
import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests.test_gpu_xent import plain, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nm.lib()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("V,up", [(5, [4]), (300, [17]), (3000, [0, 1, 2]), (700, range(0, 700, 2))])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_infinite_logits(V, up, dtype):
    """One token has a logit of +infinity at the words `up` and of -infinity at the others: its
    log sum is +infinity, whatever part of the vocabulary holds it, and its loss what lse - logit
    is.  The other tokens' results do not change."""
    W, X, y, g = problem(V, 64, 40, dtype, 3)
    W[:, 3] = -1.0
    W[list(up), 3] = 1.0
    clean, _ = nm.xent(W.cuda(), X.cuda(), y.cuda())
    down = next(v for v in range(V) if v not in up)
    for target in (list(up)[0], down):
        X[3, 9], y[9] = float("inf"), target
        loss, lse = nm.xent(W.cuda(), X.cuda(), y.cuda())
        assert float(lse[9]) == float("inf")
        assert loss[9].isnan() if target != down else float(loss[9]) == float("inf")
        others = [t for t in range(40) if t != 9]
        assert torch.equal(loss[others], clean[others])
        # P is 0 at the words of -infinity: their rows of dW see 0 x infinity at feature 3 alone
        dW, dX = (t.cpu() for t in nm.xent_grad(W.cuda(), X.cuda(), y.cuda(), lse, g.cuda()))
        want = plain(W, X, y, g)
        assert torch.equal(dW.isnan(), want["dW"].isnan())
        assert torch.equal(dX.isnan(), want["dX"].isnan())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_left_out_tokens_have_no_gradient_whatever_W_holds(dtype, bad):
    """A word whose row of W is not finite spoils the live tokens, not those that are left out."""
    W, X, y, g = problem(300, 64, 40, dtype, 11)
    W[7] = bad
    y[5], y[30] = -100, 300
    loss, lse = nm.xent(W.cuda(), X.cuda(), y.cuda())
    _, dX = nm.xent_grad(W.cuda(), X.cuda(), y.cuda(), lse, g.cuda())
    left = (y < 0) | (y >= 300)
    assert (loss.cpu()[left] == 0).all() and (dX.cpu()[:, left] == 0).all()
    assert dX.cpu()[:, ~left].isnan().any()


def uneven(V, K, T, small, seed):
    """Positive, nearly equal logits: each word's probability is about 1 / V, and dX sums V of them.
    Every second token's gout is `small` times the others'."""
    gen = torch.Generator().manual_seed(seed)
    W = (1 + torch.rand(V, K, generator=gen, dtype=torch.float64)).half()
    X = (torch.randn(K, T, generator=gen, dtype=torch.float64) * 0.1).half()
    y = torch.randint(0, V, (T,), generator=gen)
    gout = torch.full((T,), 2.0 ** 12) * (1 + torch.rand(T, generator=gen)) / 2
    gout[::2] *= small
    return W, X, y, gout


@pytest.mark.parametrize("V,K,T", [(8000, 64, 24), (8000, 65, 77), (20000, 256, 300)])
@pytest.mark.parametrize("small", [2.0 ** -8, 2.0 ** -15, 2.0 ** -21, 2.0 ** -25])
def test_uneven_gout(V, K, T, small):
    """fp16: a token's column of dX is as accurate beside tokens of far larger gout as alone, and dW
    loses nothing that counts beside its largest terms.

    Per element, with test_gpu_xent's u, e and magnitudes.  P is held at 2^0 or more for a
    probability of 1, so an entry is off by at most u of itself or 2^-25 g: V of those add up to
    2^-25 g sum |W|.  In dW a token's X may be brought down so far that 2^-25 of it is lost, 2^-39
    of the largest g beside a P of 1 (sum of |P| over a row's tokens), and P's own least numbers
    are 2^-39 of the largest g beside |X|.  The results are rounded to fp16, 2^-25 at the least."""
    W, X, y, gout = uneven(V, K, T, small, V + K + T)
    W, X, y, gout = (t.cuda() for t in (W, X, y, gout))
    _, lse = nm.xent(W, X, y)
    dW, dX = (t.double() for t in nm.xent_grad(W, X, y, lse, gout))
    with torch.device("cuda"):
        want = plain(W, X, y, gout)
    u, g = 2.0 ** -11, gout.double()
    top = want["l"].abs().max()
    lse_off = 2 * want["dl"].max() + (V / 32 + 64) * 2.0 ** -24 + 2.0 ** -21 * (1 + top)
    e = float(2 * lse_off) + (max(V, T) + 64) * 2.0 ** -24
    w, x = W.double().abs(), X.double().abs()
    bound = ((u + e) * want["mX"] * (1 + u) + u * want["dX"].abs()
             + 2.0 ** -25 * g * w.sum(0)[:, None] + 2.0 ** -25)
    off = (dX - want["dX"]).abs()
    assert (off <= bound).all(), float((off / bound).max())
    gmax = g.abs().max()
    bound = ((u + e) * want["mW"] * (1 + u) + u * want["dW"].abs() + 2.0 ** -25
             + 2.0 ** -39 * (want["P"].sum(1)[:, None] + gmax * x.sum(1)))
    off = (dW - want["dW"]).abs()
    assert (off <= bound).all(), float((off / bound).max())


def test_not_finite_gout_stays_with_its_token():
    """An infinite or NaN gout spoils its own token's column; the others keep their accuracy."""
    W, X, y, gout = uneven(8000, 64, 24, 2.0 ** -25, 1)
    W, X, y, gout = (t.cuda() for t in (W, X, y, gout))
    _, lse = nm.xent(W, X, y)
    _, clean = nm.xent_grad(W, X, y, lse, gout)
    gout[3], gout[8] = float("inf"), float("nan")
    _, dX = nm.xent_grad(W, X, y, lse, gout)
    assert dX[:, 8].isnan().all() and not dX[:, 3].isfinite().any()
    keep = [t for t in range(24) if t not in (3, 8)]
    off = (dX[:, keep].double() - clean[:, keep].double()).abs()
    # each side: P off by 2^-11 of itself (magnitudes sum to 3 g) and the least numbers, 2^-25 g sum
    # W = 2^-11 g, and the result's rounding, 2^-11 of it or 2^-25
    assert (off <= 2.0 ** -8 * gout[keep].double() + 2.0 ** -10 * clean[:, keep].double().abs()
            + 2.0 ** -24).all()


def test_shifted_targets():
    """A view that starts at any entry (target = tokens[1:]) is taken as it stands."""
    W, X, y, g = (t.cuda() for t in problem(300, 64, 40, torch.bfloat16, 13))
    loss, lse = nm.xent(W, X, y)
    want = nm.xent_grad(W, X, y, lse, g)
    tokens = torch.cat([y[:1], y])
    lse1, g1 = (torch.cat([t.new_zeros(3), t])[3:] for t in (lse, g))
    assert tokens[1:].data_ptr() % 16 and lse1.data_ptr() % 16 and g1.data_ptr() % 16
    again = nm.xent(W, X, tokens[1:])
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    for a, b in zip(nm.xent_grad(W, X, tokens[1:], lse1, g1), want):
        assert torch.equal(a, b)
