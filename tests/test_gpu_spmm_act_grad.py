"""spmm_act_grad against the formula in 64 bits and against differences of the forward pass."""
import math

import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests import act_ref as ref
from tests.test_gpu_spmm_act import DT, inputs

pytestmark = pytest.mark.gpu


def run(R, K, T, n, m, dtype, layout, act, want=("dW", "dX", "dbias", "dZ"), seed=0):
    values, meta, X, W, _ = inputs(R, K, T, n, m, dtype, layout, seed)
    gen = torch.Generator().manual_seed(seed + 7)
    Z = (torch.randn(R, T, generator=gen) * 2).to(DT[dtype])
    dY = torch.randn(R, T, generator=gen).to(DT[dtype])
    expect = ref.gradient(W, X.cpu(), None if act == "none" else Z, dY, act, DT[dtype])
    got = nm.spmm_act_grad(values, meta, X, dY.cuda(), None if act == "none" else Z.cuda(), n, m,
                           act=act, layout=layout, rows=R, want=want)
    for name, g in zip(want, got):
        assert g.dtype == (torch.float32 if name == "dbias" else DT[dtype])
        ref.check(g, *expect[name], name)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R,T", [(128, 64), (100, 33)])
def test_activations(act, dtype, R, T):
    run(R, 192, T, 2, 4, dtype, "blocked", act)


@pytest.mark.parametrize("n,m,K", [(2, 4, 128), (1, 2, 64), (4, 8, 320), (1, 4, 116), (2, 4, 100),
                                   (3, 8, 8), (2, 4, 4)])
@pytest.mark.parametrize("T", [1, 65])
def test_patterns_and_widths(n, m, K, T):
    run(70, K, T, n, m, "bf16", "rows", "silu")
    if K % 64 == 0:
        run(70, K, T, n, m, "bf16", "blocked", "silu")


@pytest.mark.parametrize("R,K,T", [(1, 64, 1), (64, 64, 64), (65, 64, 63), (1000, 768, 333),
                                   (2100, 64, 700), (64, 2048, 8), (40, 64, 5000), (4096, 64, 9),
                                   (2048, 1024, 512), (700, 1984, 1000)])
def test_sizes(R, K, T):
    run(R, K, T, 2, 4, "fp16", "blocked", "gelu")


@pytest.mark.parametrize("want", [("dZ",), ("dbias",), ("dW",), ("dX",), ("dX", "dW"),
                                  ("dbias", "dZ"), ("dZ", "dW")])
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("R,T", [(64, 128), (70, 45)])
def test_wanted_parts(want, act, R, T):
    run(R, 128, T, 2, 4, "bf16", "blocked", act, want)


def test_parts_need_only_their_inputs():
    dY = torch.randn(30, 40).to(torch.bfloat16).cuda()
    X = torch.randn(64, 40).to(torch.bfloat16).cuda()
    dz, db = nm.spmm_act_grad(None, None, None, dY, want=("dZ", "dbias"))
    assert torch.equal(dz, dY)
    (dw,) = nm.spmm_act_grad(None, None, X, dY, want=("dW",))
    expect = ref.gradient(None, X.cpu(), None, dY.cpu(), "none", torch.bfloat16)
    ref.check(dw, *expect["dW"], "dW")
    ref.check(db, *expect["dbias"], "dbias")


def test_no_tokens_give_zeros():
    values, meta, X, _, _ = inputs(32, 64, 4, 2, 4, "bf16", "blocked")
    empty = torch.zeros(32, 0, dtype=torch.bfloat16, device="cuda")
    dW, dX, db = nm.spmm_act_grad(values, meta, X[:, :0].contiguous(), empty, layout="blocked", rows=32)
    assert bool((dW == 0).all()) and dX.shape == (64, 0) and bool((db == 0).all())


def test_neither_tokens_nor_columns_nor_rows():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    torch.full((7,), 9.0, device="cuda")  # (what an allocation may find)
    (db,) = nm.spmm_act_grad(None, None, None, torch.zeros(7, 0, **bf), want=("dbias",))
    dW, db2 = nm.spmm_act_grad(None, None, torch.zeros(0, 0, **bf), torch.zeros(7, 0, **bf),
                               want=("dW", "dbias"))
    assert db.tolist() == [0.0] * 7 == db2.tolist() and dW.shape == (7, 0)
    values, meta = nm.compress(torch.zeros(0, 64, **bf), 2, 4)
    dW, dX, db = nm.spmm_act_grad(values, meta, torch.ones(64, 5, **bf), torch.zeros(0, 5, **bf))
    assert dW.shape == (0, 64) and bool((dX == 0).all()) and db.shape == (0,)


def test_infinite_columns_stay_where_they_are():
    """Z of +-infinity has slope 1 or 0; a masked (relu) entry of dY may hold anything."""
    Z = torch.tensor([[math.inf, -math.inf, 1e30, -1e30, 0.0]]).to(torch.bfloat16).cuda()
    dY = torch.full_like(Z, 2.0)
    for act, first in (("relu", 2.0), ("silu", 2.0), ("gelu", 2.0), ("gelu_tanh", 2.0)):
        (dZ,) = nm.spmm_act_grad(None, None, None, dY, Z, act=act, want=("dZ",))
        assert dZ[0, :4].tolist() == [first, 0.0, first, 0.0], act
    dY[0, 1] = math.inf
    dY[0, 3] = math.nan
    (dZ,) = nm.spmm_act_grad(None, None, None, dY, Z, act="relu", want=("dZ",))
    assert dZ[0].tolist() == [2.0, 0.0, 2.0, 0.0, 0.0]


@pytest.mark.parametrize("act", ref.ACTS)
def test_against_differences(act):
    """The loss sum(dY * Y) of an fp32 product, X moved by +-h in one direction: the 64-bit formula's
    directional derivative, which the kernels are held to above, is the difference quotient's limit."""
    R, K, T = 48, 64, 20
    values, meta, X, W, Xd = inputs(R, K, T, 2, 4, "fp16", "blocked", seed=3)
    gen = torch.Generator().manual_seed(5)
    b = torch.randn(R, generator=gen).double()
    dY = torch.randn(R, T, generator=gen).to(torch.float16)
    way = torch.randn(K, T, generator=gen).double()
    h = 1e-5
    # a kink of relu within h of any sum would spoil the quotient
    z = W @ Xd + b[:, None]
    loss = lambda x: float((ref.act(W @ x + b[:, None], act) * dY.double()).sum())
    quotient = (loss(Xd + h * way) - loss(Xd - h * way)) / (2 * h)
    Z = z.to(torch.float16)
    (dX,) = nm.spmm_act_grad(values, meta, X, dY.cuda(), Z.cuda(), act=act, layout="blocked", rows=R,
                             want=("dX",))
    got = float((dX.double().cpu() * way).sum())
    # Z in fp16 moves the slope by at most 2^-11 |Z| times its own slope (below 2), dZ and dX round
    # once each: relative 2^-11 of each term
    dz = dY.double() * ref.slope(z, act)
    size = float((way.abs() * (W.abs().t() @ (dY.double().abs() * (z.abs() + 1)))).sum())
    assert abs(got - quotient) <= 4 * 2.0 ** -11 * size, (got, quotient)
    assert dz.shape == (R, T)
