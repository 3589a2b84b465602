"""Cross entropy of a large vocabulary and its gradient against plain 64-bit implementations.

Tolerances, per element.  A logit is an fp32 sum of K exact products: |d l| <= K 2^-24 sum |w x|.
lse and the target's logit move by at most the largest of those, and the exponentials' sum adds
(V / 32 + 64) 2^-24 relative at most, besides a few 2^-22 for exp2 and log2 on numbers of their size.
P is rounded to the inputs' type (relative u), and the error of l - lse enters it as a factor, so
  |d dX| <= (u + e) W^T |P'| + u |dX|,  |d dW| <= (u + e) |P'| X^T + u |dW|,
with P' = (softmax + one-hot) |g| over |W|, |X|, and e the relative error of the exponentials plus
the fp32 sums' (length 2^-24); an fp16 P keeps numbers down to 2^-24 of its largest.
"""
import pytest
import torch

import masking_sparse_gemm_amd as nm

pytestmark = pytest.mark.gpu

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nm.lib()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def problem(V, K, T, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(V + 31 * K + 977 * T + seed)
    W = (torch.randn(V, K, generator=g, dtype=torch.float64) * scale / max(1, K) ** 0.5).to(dtype)
    X = torch.randn(K, T, generator=g, dtype=torch.float64).to(dtype)
    y = torch.randint(0, V, (T,), generator=g)
    if T > 2:
        y[1] = -100
        y[T - 1] = V - 1
    gout = torch.rand(T, generator=g) / T
    return W, X, y, gout


def plain(W, X, y, gout):
    w, x, g = W.double(), X.double(), gout.double()
    V, T = w.shape[0], x.shape[1]
    l = w @ x
    lse = torch.logsumexp(l, 0)
    live = (y >= 0) & (y < V)
    at = y.clamp(0, V - 1)[None]
    loss = torch.where(live, lse - l.gather(0, at)[0], torch.zeros(T, dtype=torch.float64))
    soft = torch.exp(l - lse)
    hot = torch.zeros_like(soft).scatter_(0, at, 1.0)
    gl = torch.where(live, g, torch.zeros_like(g))
    P, Pabs = (soft - hot) * gl, (soft + hot) * gl.abs()
    xl = torch.where(live[None], x, torch.zeros_like(x))
    return dict(l=l, lse=lse, loss=loss, dW=P @ xl.t(), dX=w.t() @ P, P=Pabs, live=live,
                mW=Pabs @ xl.abs().t(), mX=w.abs().t() @ Pabs,
                dl=w.shape[1] * 2.0 ** -24 * (w.abs() @ x.abs()).amax(0), gmax=gl.abs().max())


def check(V, K, T, dtype, seed=0, scale=1.0, grad=True, data=None):
    W, X, y, gout = data or problem(V, K, T, dtype, seed, scale)
    want = plain(W, X, y, gout)
    Wd, Xd, yd = W.cuda(), X.cuda(), y.cuda()
    loss, lse = nm.xent(Wd, Xd, yd)
    top = want["l"].abs().amax(0)
    tol = 2 * want["dl"] + (V / 32 + 64) * 2.0 ** -24 + 2.0 ** -21 * (1 + top)
    assert ((lse.cpu().double() - want["lse"]).abs() <= tol).all()
    assert ((loss.cpu().double() - want["loss"]).abs() <= 2 * tol).all()
    assert (loss.cpu()[~want["live"]] == 0).all()
    if not grad:
        return
    dW, dX = nm.xent_grad(Wd, Xd, yd, lse, gout.cuda())
    assert dW.dtype == dX.dtype == dtype and dW.shape == W.shape and dX.shape == X.shape
    u = ROUND[dtype]
    e = float(2 * tol.max()) + (max(V, T) + 64) * 2.0 ** -24
    # an fp16 P below 2^-14 of ~2^13 keeps 2^-25 absolute, of at most that many terms
    small = 2.0 ** -37 * float(want["gmax"]) if dtype == torch.float16 else 0.0
    tiny = 2.0 ** -25 if dtype == torch.float16 else 1e-30
    for got, name, mag, n in ((dW, "dW", "mW", X.double().abs().sum(1)[None]),
                              (dX, "dX", "mX", W.double().abs().sum(0)[:, None])):
        err = (got.cpu().double() - want[name]).abs()
        bound = (u + e) * want[mag] * (1 + u) + u * want[name].abs() + small * n + tiny
        assert (err <= bound).all(), (name, float((err / bound).max()))
    # a token left out adds nothing to its column
    assert (dX.cpu()[:, ~want["live"]] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V,K,T", [(1, 1, 1), (2, 8, 3), (7, 64, 5), (130, 64, 1), (257, 128, 64),
                                   (1000, 72, 65), (513, 100, 33), (300, 320, 200),
                                   (2048, 65, 130), (63, 256, 300), (640, 192, 129)])
def test_small_and_odd_sizes(V, K, T, dtype):
    check(V, K, T, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_large_tiles(dtype):
    """Enough tiles for the 256 x 256 kernels of every product, with ragged ends."""
    check(8200, 2112, 1100, dtype)


def test_pieces_of_the_vocabulary():
    """More tokens than one piece of the vocabulary holds: dX adds up over pieces."""
    check(1500, 64, 45000, torch.bfloat16)


@pytest.mark.parametrize("scale", [0.01, 8.0, 40.0])
def test_flat_and_peaked(scale):
    check(700, 128, 96, torch.bfloat16, seed=3, scale=scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("factor", [2.0 ** -20, 1.0, 4096.0])
def test_size_of_gout(dtype, factor):
    """The upstream gradient's size costs no accuracy, up to the results' own range."""
    W, X, y, g = problem(500, 64, 80, dtype, 4)
    if dtype == torch.float16 and factor < 1:
        X = X * 256   # keeps dW within fp16's normal numbers
        W = W / 256
    check(500, 64, 80, dtype, data=(W, X, y, g * factor))


def test_negative_and_zero_gout():
    W, X, y, g = problem(500, 64, 80, torch.bfloat16, 5)
    g[::3] = 0
    g[1::3] *= -1
    check(500, 64, 80, torch.bfloat16, data=(W, X, y, g))


def test_every_token_left_out():
    W, X, _, g = problem(100, 64, 16, torch.bfloat16)
    for y in (torch.full((16,), -1), torch.full((16,), 100)):
        loss, lse = nm.xent(W.cuda(), X.cuda(), y.cuda())
        assert (loss == 0).all()
        dW, dX = nm.xent_grad(W.cuda(), X.cuda(), y.cuda(), lse, g.cuda())
        assert (dW == 0).all() and (dX == 0).all()


def test_what_is_left_out_may_hold_anything():
    """NaN and infinities in the columns of tokens left out change nothing."""
    W, X, y, g = problem(300, 64, 40, torch.bfloat16, 7)
    y[5] = y[17] = -100
    bad = X.clone()
    bad[:, 5] = float("nan")
    bad[3, 17] = float("inf")
    gb = g.clone()
    gb[5] = float("nan")
    out = []
    for x, gg in ((X, g), (bad, gb)):
        loss, lse = nm.xent(W.cuda(), x.cuda(), y.cuda())
        out.append((loss, *nm.xent_grad(W.cuda(), x.cuda(), y.cuda(), lse, gg.cuda())))
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_not_finite_logits():
    """A NaN logit makes its token's loss NaN and no other's; a row of W of -inf logits (a word
    that cannot occur) has probability 0."""
    W, X, y, g = problem(300, 64, 40, torch.bfloat16, 8)
    X[:, 9] = float("nan")
    y[9] = 3
    loss, lse = nm.xent(W.cuda(), X.cuda(), y.cuda())
    assert loss[9].isnan() and loss.isnan().sum() == 1
    X = X.abs().nan_to_num(1.0)
    W[4] = float("-inf")
    y[y == 4] = 5
    want = plain(W, X, y, g)
    loss, lse = nm.xent(W.cuda(), X.cuda(), y.cuda())
    assert torch.allclose(loss.cpu().double(), want["loss"], atol=1e-4)


def test_gradient_against_differences():
    """sum(gout loss) along a direction, by central differences of the 64-bit loss."""
    W, X, y, g = problem(200, 64, 48, torch.bfloat16, 9)
    _, lse = nm.xent(W.cuda(), X.cuda(), y.cuda())
    dW, dX = (t.cpu().double() for t in nm.xent_grad(W.cuda(), X.cuda(), y.cuda(), lse, g.cuda()))
    gen = torch.Generator().manual_seed(1)
    aw = torch.randn(W.shape, generator=gen, dtype=torch.float64)
    ax = torch.randn(X.shape, generator=gen, dtype=torch.float64)

    def total(h):
        return float((plain(W.double() + h * aw, X.double() + h * ax, y, g)["loss"] * g.double()).sum())

    h = 1e-4
    want = (total(h) - total(-h)) / (2 * h)
    got = float((dW * aw).sum() + (dX * ax).sum())
    # entries are off by up to 2^-7 of theirs, in random directions
    spread = float(((dW * aw) ** 2).sum() + ((dX * ax) ** 2).sum()) ** 0.5
    assert abs(got - want) <= 8 * 2.0 ** -7 * spread + 1e-7


def test_repeatable_and_on_the_current_stream():
    W, X, y, g = (t.cuda() for t in problem(3000, 256, 500, torch.bfloat16, 10))
    loss, lse = nm.xent(W, X, y)
    first = nm.xent_grad(W, X, y, lse, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        W2 = W * 1
        loss2, lse2 = nm.xent(W2, X, y)
        second = nm.xent_grad(W2, X, y, lse2, g)
    side.synchronize()
    for a, b in zip((loss, lse, *first), (loss2, lse2, *second)):
        assert torch.equal(a, b)


def test_empty():
    W = torch.ones(5, 64, dtype=torch.bfloat16, device="cuda")
    X = torch.ones(64, 0, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(0, dtype=torch.int64, device="cuda")
    loss, lse = nm.xent(W, X, y)
    assert loss.shape == lse.shape == (0,)
    dW, dX = nm.xent_grad(W, X, y, lse, loss)
    assert (dW == 0).all() and dX.shape == (64, 0)
    # no features: every logit is 0
    W, X = W[:, :0].contiguous(), torch.ones(0, 3, dtype=torch.bfloat16, device="cuda")
    loss, lse = nm.xent(W, X, torch.tensor([0, 4, -1], device="cuda"))
    assert torch.allclose(lse.cpu(), torch.full((3,), 5.0).log())
    assert torch.allclose(loss.cpu(), torch.tensor([5.0, 5.0, 1.0]).log())
