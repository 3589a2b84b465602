"""spmm_act_grad in fp16 at the ends of the type's range: slopes that leave nothing of a small dY in 16
bits, relu's square past 65504, rows and tokens far smaller than others."""
import math

import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests import act_ref as ref
from tests.test_gpu_lm_graph import randn
from tests.test_gpu_more_graph import capture
from tests.test_gpu_spmm_act import inputs

pytestmark = pytest.mark.gpu

HALF = torch.float16
# The largest |dY| (relu2: |dZ|) of a row or column is held in 2^14 .. 2^15, and fp16's smallest half step
# is 2^-25.
LOST = 2.0 ** -39


def expected(W, X, Z, dY, act):
    """{name: (value, bound)}: a product's operand is off by half a step of the entry, or of the smallest
    that its row (dW) or column (dX) still holds."""
    z, dy = Z.double(), dY.double()
    slope = ref.slope(z, act)
    dz = dy * slope
    off = ref.SLOPE_OFF * dy.abs() * (1 + (z.abs() if act == "relu2" else 0))
    # silu's s (1 + z (1 - s)): s's exponent z log2(e) rounds to 2^-24 of itself, which at z = -9 is 6e-7 of s,
    # and the few other steps round once each, to 2^-18 of both factors' sizes at most
    if act == "silu":
        off = torch.minimum(off, 2.0 ** -18 * dy.abs() * torch.sigmoid(z) * (1 + z.abs()))
    if act == "relu2":  # two products
        off = 2 * ref.F32 * dz.abs()
    entry = off + ref.HALF[HALF] * (dz.abs() + off)
    x, w = X.double(), W.double()
    R, T = dz.shape
    res = {}
    size = dz.abs() if act == "relu2" else dy.abs()
    row = entry + LOST * size.amax(1, keepdim=True)
    v = dz @ x.t()
    b = row @ x.abs().t() + ref.sum_bound(T, dz.abs() @ x.abs().t())
    res["dW"] = (v, (b + ref.rounding(v, HALF)) * (1 + 2 * ref.HALF[HALF]))
    col = entry + LOST * size.amax(0, keepdim=True)
    v = w.t() @ dz
    b = w.abs().t() @ col + ref.sum_bound(R, w.abs().t() @ dz.abs())
    res["dX"] = (v, (b + ref.rounding(v, HALF)) * (1 + 2 * ref.HALF[HALF]))
    res["dbias"] = (dz.sum(1), off.sum(1) + ref.sum_bound(T, dz.abs().sum(1)))
    res["dZ"] = (dz, (off + ref.rounding(dz, HALF)) * (1 + 2 * ref.HALF[HALF]))
    return res


def check(got, v, b, what):
    """Within its bound, where a result past fp16's largest number is infinite, and one whose bound spans the
    border (65520, half a step past it) may be either."""
    top = 65520.0
    border = (v.abs() + b >= top) & (v.abs() - b < top)
    v = torch.where(v.abs() - b >= top, v.sign() * math.inf, v)
    g = got.double().cpu()
    near = torch.where(g.abs() == math.inf, torch.full_like(g, top), g.abs()) * g.sign()
    assert bool(((near - v).abs() <= b)[border & v.isfinite()].all()), what
    ref.check(got, torch.where(border, g, v), b, what)


def run(R, K, T, act, Z, dY, x_scale=1.0, want=("dW", "dX", "dbias")):
    values, meta, X, W, _ = inputs(R, K, T, 2, 4, "fp16", "blocked")
    X = (X.float() * x_scale).to(HALF)
    got = nm.spmm_act_grad(values, meta, X, dY.cuda(), Z.cuda(), act=act, layout="blocked", rows=R, want=want)
    expect = expected(W, X.cpu(), Z, dY, act)
    for name, g in zip(want, got):
        check(g, *expect[name], name) if name != "dbias" else ref.check(g, *expect[name], name)
    return dict(zip(want, got)), expect


def normal(R, T, seed):
    return torch.randn(R, T, generator=torch.Generator().manual_seed(seed))


# sizes: one chunk of rows for the columns' largest and many, whole steps and ragged, split sums
SIZES = [(64, 64, 64), (70, 128, 333), (3000, 64, 600), (1025, 192, 40), (1500, 64, 3000)]


@pytest.mark.parametrize("R,K,T", SIZES)
def test_slopes_that_leave_nothing_of_a_small_gradient(R, K, T):
    """silu's slope at -6 .. -9 is 2^-6 .. 2^-10: on a dY of 2^-21 that is below fp16's 2^-25, but a sum of
    T of them times X is not."""
    Z = (-7.5 + normal(R, T, 1).clamp(-1.5, 1.5)).to(HALF)
    dY = (normal(R, T, 2) * 2.0 ** -21).to(HALF)
    got, expect = run(R, K, T, "silu", Z, dY, x_scale=1000.0)
    if T >= 333:  # there the unscaled rounding would have lost everything
        assert float(expect["dW"][0].abs().max()) > 2.0 ** -20
        assert float(got["dW"].abs().max()) > 0


@pytest.mark.parametrize("R,K,T", SIZES)
@pytest.mark.parametrize("want", [("dW",), ("dX",), ("dX", "dbias", "dW")])
def test_squares_past_the_largest_number(R, K, T, want):
    """2 Z dY = 120000 in one place: finite results in fp32, so finite here."""
    Z, dY = (normal(R, T, 3) * 0.01).to(HALF), (normal(R, T, 4) * 0.01).to(HALF)
    Z[R // 2, T // 3], dY[R // 2, T // 3] = 300.0, 200.0
    got, expect = run(R, K, T, "relu2", Z, dY, x_scale=0.01, want=want)
    for name in want:
        fits = expect[name][0].abs() < 60000
        assert bool(got[name].cpu()[fits].isfinite().all())
    assert not bool((Z.double() * 2 * dY.double()).abs().max() < 65504)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "relu2"])
@pytest.mark.parametrize("R,K,T", SIZES)
def test_rows_and_tokens_far_smaller_than_others(act, R, K, T):
    """A row 2^-16 of the others keeps its accuracy in dW, a token 2^-14 of them in dX."""
    Z = (normal(R, T, 5) + 1).to(HALF)
    dY = normal(R, T, 6) * 1000
    dY[R // 3] *= 2.0 ** -16
    dY[:, T // 2] *= 2.0 ** -14
    run(R, K, T, act, Z, dY.to(HALF), x_scale=1e-3)


def test_largest_of_a_row_and_of_a_column_anywhere():
    """The largest entry of a row and of a column in each place that a work-item has, one at a time in
    a matrix of small ones: none of them leaves the type's range."""
    R, K, T = 1100, 64, 130
    values, meta, X, W, _ = inputs(R, K, T, 2, 4, "fp16", "blocked")
    Z = torch.full((R, T), 100.0).to(HALF)
    dY = torch.full((R, T), 2.0 ** -10).to(HALF)
    at = torch.arange(R) * 7 % T
    dY[torch.arange(R), at] = 60000.0      # every row has one, every column some
    got = nm.spmm_act_grad(values, meta, (X.float() * 1e-4).to(HALF), dY.cuda(), Z.cuda(), act="relu2",
                           layout="blocked", rows=R, want=("dW",))
    expect = expected(W, (X.float() * 1e-4).to(HALF).cpu(), Z, dY, "relu2")
    ref.check(got[0], *expect["dW"], "dW")


def test_infinities_and_nan_stay_in_their_row_and_column():
    R, K, T = 100, 64, 70
    values, meta, X, W, _ = inputs(R, K, T, 2, 4, "fp16", "blocked")
    Z, dY = normal(R, T, 7).to(HALF), normal(R, T, 8).to(HALF)
    clean = nm.spmm_act_grad(values, meta, X, dY.cuda(), Z.cuda(), act="gelu", layout="blocked", rows=R)
    dY[5, 9], dY[60, 33] = math.inf, math.nan
    dW, dX, db = nm.spmm_act_grad(values, meta, X, dY.cuda(), Z.cuda(), act="gelu", layout="blocked", rows=R)
    rows = [r for r in range(R) if r not in (5, 60)]
    cols = [t for t in range(T) if t not in (9, 33)]
    assert torch.equal(dW[rows], clean[0][rows]) and torch.equal(dX[:, cols], clean[1][:, cols])
    assert not bool(dW[[5, 60]].isfinite().any()) and bool(db[[5, 60]].isfinite().logical_not().all())


def test_all_zeros():
    R, K, T = 65, 64, 33
    values, meta, X, _, _ = inputs(R, K, T, 2, 4, "fp16", "blocked")
    zero = torch.zeros(R, T, dtype=HALF, device="cuda")
    for g in nm.spmm_act_grad(values, meta, X, zero, zero, act="silu", layout="blocked", rows=R, want=nm.GRADS):
        assert bool((g == 0).all())


@pytest.mark.parametrize("want", [("dZ",), ("dZ", "dW"), ("dX", "dZ"), ("dbias", "dZ", "dX", "dW")])
@pytest.mark.parametrize("R,T", [(64, 128), (70, 45)])
def test_wanted_parts(want, R, T):
    run(R, 128, T, "gelu", normal(R, T, 9).to(HALF), normal(R, T, 10).to(HALF), want=want)


@pytest.mark.parametrize("R,T", [(256, 128), (2001, 77)])
def test_replays_of_a_graph(R, T):
    values, meta = nm.compress(randn(R, 512, seed=9).half() * 512 ** -0.5, 2, 4, layout="blocked")
    call = lambda x, z, dy: nm.spmm_act_grad(values, meta, x, dy, z, act="gelu", layout="blocked", rows=R,
                                             want=nm.GRADS)
    fresh = lambda seed: (randn(512, T, seed=seed).half(), randn(R, T, seed=seed + 1).half(),
                          randn(R, T, seed=seed + 2).half() * 2.0 ** (seed % 5 - 8))
    state = fresh(1)
    graph, out = capture(call, state)
    for replay in range(4):
        new = fresh(10 + replay)
        for a, b in zip(state, new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, call(*new)):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, HALF])
@pytest.mark.parametrize("R,K,layout", [(70, 128, "blocked"), (70, 100, "rows"), (1, 64, "blocked"),
                                        (2051, 2112, "blocked")])
def test_an_infinity_in_the_last_row_of_W(dtype, R, K, layout):
    """Rows that make W whole steps hold zeros: the last one's infinity is infinite in dX, not NaN, and
    reaches no other row of dX."""
    T = 33
    w = torch.randn(R, K, generator=torch.Generator().manual_seed(1)).to(dtype)
    w[R - 1, 4] = math.inf
    dY = (normal(R, T, 11).abs() + 0.5).to(dtype)
    dY[:, ::2] *= -1
    values, meta = nm.compress(w.cuda(), 2, 4, layout=layout)
    X = torch.zeros(K, T, dtype=dtype, device="cuda")
    (dX,) = nm.spmm_act_grad(values, meta, X, dY.cuda(), layout=layout, rows=R, want=("dX",))
    assert torch.equal(dX[4].cpu(), torch.where(dY[R - 1] > 0, math.inf, -math.inf).to(dtype))
    assert bool(dX[[k for k in range(K) if k != 4]].isfinite().all())
