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
