"""spmm_act against a 64-bit reference: every type, pattern, layout and tile, sizes from one token
on, odd ones, and the epilogue's parts alone and together."""
import math
import os

import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests import act_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn,
      "int8": torch.int8}
EIGHT = ("fp8", "int8")


def inputs(R, K, T, n, m, dtype, layout, seed=0):
    """(values, meta, X, dense W in 64 bits, X in 64 bits)."""
    gen = torch.Generator().manual_seed(seed)
    w, x = torch.randn(R, K, generator=gen), torch.randn(K, T, generator=gen)
    if dtype == "int8":
        w, x = (w * 40).round().clamp(-128, 127), (x * 40).round().clamp(-128, 127)
    else:
        w = w / math.sqrt(max(1, K * n / m)) if dtype != "fp8" else w
    w, x = w.to(DT[dtype]).cuda(), x.to(DT[dtype]).cuda()
    values, meta = nm.compress(w, n, m, layout=layout)
    dense = nm.decompress(values, meta, n, m, K, layout=layout, rows=R)
    return values, meta, x, dense.double().cpu(), x.double().cpu()


def run(R, K, T, n, m, dtype, layout, act, bias, residual, keep, y, seed=0):
    values, meta, X, W, Xd = inputs(R, K, T, n, m, dtype, layout, seed)
    gen = torch.Generator().manual_seed(seed + 100)
    y_dt = DT[y]
    b = torch.randn(R, generator=gen) if bias else None
    r = torch.randn(R, T, generator=gen).to(y_dt) if residual else None
    s = None
    sums = W @ Xd
    off = ref.sum_bound(K // m * n, W.abs() @ Xd.abs())
    if dtype == "fp8":  # the instruction's runs of 16: 7 2^(e - 13) each, 2^e up to twice its largest
        off = off + 7 * 2.0 ** -12 * (W.abs() @ Xd.abs())
    if dtype in EIGHT:
        s = (torch.rand(R, generator=gen) + 0.5) / (40 * 40 if dtype == "int8" else 1) / math.sqrt(K)
        sums, off = sums * s.double()[:, None], off * s.double()[:, None]
        off = off + 2 * ref.F32 * sums.abs()
    cuda = lambda t: None if t is None else t.cuda()
    got = nm.spmm_act(values, meta, X, n, m, bias=cuda(b), act=act, residual=cuda(r), scale=cuda(s),
                      keep=keep, out_dtype=y_dt, layout=layout, rows=R)
    Y, Z = got if keep else (got, None)
    wy, by, wz, bz = ref.epilogue(sums, off, b, act, r, y_dt, DT[dtype] if keep else None)
    assert Y.dtype == y_dt
    ref.check(Y, wy, by, "Y")
    if keep:
        assert Z.dtype == DT[dtype]
        ref.check(Z, wz, bz, "Z")


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype,y", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"),
                                     ("fp32", "fp32"), ("fp8", "bf16"), ("fp8", "fp32"),
                                     ("int8", "fp16"), ("int8", "fp32")])
def test_types_and_activations(act, dtype, y):
    run(100, 256, 48, 2, 4, dtype, "blocked", act, True, True, dtype not in EIGHT, y)


@pytest.mark.parametrize("n,m", [(2, 4), (1, 2), (4, 8), (1, 4), (3, 8), (2, 2)])
@pytest.mark.parametrize("layout", ["rows", "blocked"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32", "int8", "fp8"])
def test_patterns_and_layouts(n, m, layout, dtype):
    if layout == "blocked" and dtype in EIGHT and (16 * n // m) % 4:
        pytest.skip("bytes of this pattern have no blocked layout")
    run(77, 192, 33, n, m, dtype, layout, "silu", True, True, dtype not in EIGHT,
        "bf16" if dtype in EIGHT else dtype)


@pytest.mark.parametrize("R,K,T", [(1, 64, 1), (16, 64, 1), (17, 128, 3), (300, 64, 7), (129, 1024, 8),
                                   (64, 4096, 1), (257, 320, 129), (1000, 1024, 517), (5, 64, 1030),
                                   (2048, 64, 16), (33, 640, 40)])
@pytest.mark.parametrize("layout", ["rows", "blocked"])
def test_sizes(R, K, T, layout):
    run(R, K, T, 2, 4, "bf16", layout, "gelu", True, True, True, "bf16")


@pytest.mark.parametrize("n,m", [(2, 4), (1, 2), (1, 4), (4, 8)])
@pytest.mark.parametrize("layout", ["rows", "blocked"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32", "int8", "fp8"])
@pytest.mark.parametrize("R,K", [(70, 640), (1100, 2048)])
def test_one_token(n, m, layout, dtype, R, K):
    run(R, K, 1, n, m, dtype, layout, "gelu", True, True, dtype not in EIGHT,
        "fp32" if dtype in EIGHT else dtype)


# test_more_tiles.py holds the rule to every shape of a workgroup here, with X turned and as it lies
@pytest.mark.parametrize("n,m", [(2, 4), (1, 2), (1, 4), (4, 8)])
@pytest.mark.parametrize("layout", ["rows", "blocked"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32", "int8", "fp8"])
@pytest.mark.parametrize("R,K,T", [(1000, 1024, 517), (2048, 1024, 517), (256, 192, 1000), (256, 192, 2000)])
def test_thin_shapes(n, m, layout, dtype, R, K, T):
    run(R, K, T, n, m, dtype, layout, "relu", True, True, dtype not in EIGHT,
        "fp32" if dtype in EIGHT else dtype)


@pytest.mark.parametrize("n,m", [(2, 4), (1, 2), (1, 4), (4, 8)])
@pytest.mark.parametrize("K", [192, 184])
def test_infinite_columns_of_X_stay_where_they_are(n, m, K):
    """A column's numbers reach no other column, and those past the last one are no column's."""
    R, T = 77, 33
    values, meta, X, W, _ = inputs(R, K, T, n, m, "bf16", "rows")
    want = nm.spmm_act(values, meta, X, n, m)
    for t in (0, 16, 32):
        Y = X.clone()
        Y[:, t] = math.nan
        got = nm.spmm_act(values, meta, Y, n, m)
        assert bool(got[:, t].isnan().all())
        rest = [c for c in range(T) if c != t]
        assert torch.equal(got[:, rest], want[:, rest])


@pytest.mark.parametrize("n,m", [(2, 4), (1, 2), (1, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32", "int8", "fp8"])
@pytest.mark.parametrize("K", [8, 72, 148, 1020])
def test_few_tokens_of_every_type_and_any_width(n, m, dtype, K):
    run(45, K, 20, n, m, dtype, "rows", "silu", True, False, False, "fp32" if dtype in EIGHT else dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32", "int8", "fp8"])
@pytest.mark.parametrize("K", [8, 16, 72, 120, 152, 1016])
@pytest.mark.parametrize("T", [1, 20])
def test_4_of_8_of_any_width(dtype, K, T):
    run(45, K, T, 4, 8, dtype, "rows", "silu", True, False, False, "fp32" if dtype in EIGHT else dtype)


def test_bytes_without_a_scale():
    values, meta, X, W, Xd = inputs(40, 128, 24, 2, 4, "int8", "blocked")
    Y = nm.spmm_act(values, meta, X, out_dtype=torch.float32, layout="blocked", rows=40)
    assert torch.equal(Y.double().cpu(), W @ Xd)  # whole numbers below 2^24


@pytest.mark.parametrize("K", [4, 20, 100, 1004])
@pytest.mark.parametrize("T", [1, 2, 9, 64])
def test_row_layout_of_any_width(K, T):
    run(50, K, T, 2, 4, "fp16", "rows", "gelu_tanh", True, False, True, "fp32")


# sizes that the tiled kernels take (test_more_tiles.py holds the rule to it)
MANY = [(2000, 128, 2056), (2000, 128, 2061)]


@pytest.mark.parametrize("tile", ["0", "1", "2"])
@pytest.mark.parametrize("R,K,T", MANY)
def test_every_tile(tile, R, K, T, monkeypatch):
    monkeypatch.setenv("NM_SPMM_TILE", tile)
    run(R, K, T, 2, 4, "bf16", "blocked", "silu", True, True, True, "bf16")
    run(R, K, T, 1, 2, "fp16", "rows", "none", False, True, False, "fp32")


@pytest.mark.parametrize("n,m", [(2, 4), (1, 2), (4, 8), (1, 4)])
@pytest.mark.parametrize("layout", ["rows", "blocked"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32", "int8", "fp8"])
@pytest.mark.parametrize("R,K,T", MANY)
def test_many_tokens(n, m, layout, dtype, R, K, T):
    run(R, K, T, n, m, dtype, layout, "gelu", True, True, dtype not in EIGHT,
        "bf16" if dtype in EIGHT else dtype)


@pytest.mark.parametrize("dtype", ["int8", "fp8"])
def test_many_tokens_of_bytes_in_half_steps(dtype):
    run(2000, 192, 2061, 2, 4, dtype, "blocked", "relu2", True, False, False, "fp32")


@pytest.mark.parametrize("bias,residual,keep", [(b, r, k) for b in (0, 1) for r in (0, 1) for k in (0, 1)])
def test_parts(bias, residual, keep):
    run(200, 256, 72, 2, 4, "bf16", "blocked", "relu", bool(bias), bool(residual), bool(keep), "bf16")


def test_plain_call_is_spmm():
    """Both form the same sums in orders of their own, each within sum_bound, and round once."""
    values, meta, X, W, Xd = inputs(300, 512, 136, 2, 4, "bf16", "blocked")
    want = nm.spmm(values, meta, X, 2, 4, layout="blocked", rows=300).double().cpu()
    got = nm.spmm_act(values, meta, X, layout="blocked", rows=300)
    off = 2 * (ref.sum_bound(256, W.abs() @ Xd.abs()) + ref.rounding(want, torch.bfloat16))
    ref.check(got, want, off * (1 + 2 * ref.HALF[torch.bfloat16]), "Y")


def test_plain_call_is_spmm_bit_for_bit_in_the_same_kernel():
    values, meta, X, _, _ = inputs(2000, 128, 2056, 2, 4, "bf16", "blocked")
    want = nm.spmm(values, meta, X, 2, 4, layout="blocked", rows=2000)
    assert torch.equal(nm.spmm_act(values, meta, X, layout="blocked", rows=2000), want)


@pytest.mark.parametrize("T", [40, 41])
def test_onto_the_residual_in_place_and_nothing_beside_it(T):
    R, K = 70, 128
    values, meta, X, W, Xd = inputs(R, K, T, 2, 4, "bf16", "blocked")
    big = torch.full((R + 10, T), 3.0, device="cuda", dtype=torch.bfloat16)
    res = torch.randn(R, T).to(torch.bfloat16)
    big[:R] = res.cuda()
    out = nm.spmm_act(values, meta, X, residual=big[:R], out=big[:R], layout="blocked", rows=R)
    assert out.data_ptr() == big.data_ptr()
    y, b, _, _ = ref.epilogue(W @ Xd, ref.sum_bound(K // 2, W.abs() @ Xd.abs()), None, "none", res,
                              torch.bfloat16)
    ref.check(big[:R], y, b, "Y")
    assert bool((big[R:] == 3.0).all())


@pytest.mark.parametrize("act", ref.ACTS)
def test_infinities_and_nan(act):
    """A bias of +-infinity or NaN takes its row: -infinity gives 0 (plus the residual)."""
    R, K, T = 20, 64, 8
    values, meta, X, _, _ = inputs(R, K, T, 2, 4, "bf16", "blocked")
    bias = torch.zeros(R)
    bias[0], bias[1], bias[2] = math.inf, -math.inf, math.nan
    bias[3], bias[4] = 1e30, -1e30
    res = torch.ones(R, T, dtype=torch.bfloat16)
    Y, Z = nm.spmm_act(values, meta, X, bias=bias.cuda(), act=act, residual=res.cuda(), keep=True,
                       out_dtype=torch.bfloat16, layout="blocked", rows=R)
    assert bool((Y[0] == math.inf).all()) and bool((Z[0] == math.inf).all())
    assert bool((Y[1] == (-math.inf if act == "none" else 1.0)).all())
    assert bool(Y[2].isnan().all()) and bool(Z[2].isnan().all())
    assert bool((Y[3] == (math.inf if act == "relu2" else 1e30)).all() | (Y[3] > 9e29).all())
    assert bool((Y[4] < -9e29).all() if act == "none" else (Y[4] == 1.0).all())
    assert bool(Y[5:].isfinite().all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32", "int8"])
@pytest.mark.parametrize("layout", ["rows", "blocked"])
def test_no_columns_of_W_gives_the_bias(dtype, layout):
    R, T = 30, 9
    w = torch.zeros(R, 0, dtype=DT[dtype], device="cuda")
    values, meta = nm.compress(w, 2, 4, layout=layout)
    X = torch.zeros(0, T, dtype=DT[dtype], device="cuda")
    b = torch.randn(R, device="cuda")
    Y = nm.spmm_act(values, meta, X, bias=b, act="relu", out_dtype=torch.float32, layout=layout, rows=R)
    assert torch.equal(Y, b.clamp(min=0)[:, None].expand(R, T))


def test_empty_results():
    values, meta, X, _, _ = inputs(16, 64, 4, 2, 4, "bf16", "blocked")
    assert nm.spmm_act(values, meta, X[:, :0].contiguous(), layout="blocked", rows=16).shape == (16, 0)


def test_on_another_stream():
    values, meta, X, _, _ = inputs(300, 512, 33, 2, 4, "bf16", "blocked")
    want = nm.spmm_act(values, meta, X, act="gelu", layout="blocked", rows=300)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = nm.spmm_act(values, meta, X, act="gelu", layout="blocked", rows=300)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
