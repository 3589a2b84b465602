"""4-bit weights (quantize, dequantize, matvec) against plain 64-bit implementations.

Codes and scales are compared exactly: both sides round the same quotients.  Products: codes and
16-bit numbers multiply exactly, so an element's error is the fp32 summation's -- at most
K 2^-24 times the sum of the magnitudes that are added, (16 + u) |x| and 24 |x| with u <= 15 under
the group's scale -- plus the result's one rounding.
"""
import numpy as np
import pytest
import torch

import masking_sparse_gemm_amd as nm

pytestmark = pytest.mark.gpu

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nm.lib()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def weights(R, K, dtype, seed=0):
    g = torch.Generator().manual_seed(1000 * R + K + seed)
    return (torch.randn(R, K, generator=g, dtype=torch.float64) * 0.02).to(dtype)


def plain_quantize(w, group, sdtype):
    """(codes -8 .. 7 (R, C), scales (R, groups)) of a CPU matrix; the quotients in float32, as
    defined, everything else in 64 bits."""
    R, C = w.shape
    n = -(-C // group)
    codes = torch.zeros(R, C, dtype=torch.int64)
    scales = torch.zeros(R, n, dtype=sdtype)
    for i in range(n):
        part = w[:, i * group:(i + 1) * group].float()
        s = (part.abs().amax(1) / 7).to(sdtype)
        scales[:, i] = s
        q = torch.round(part / s.float()[:, None])
        q = torch.where(torch.isnan(q) | (s.float() == 0)[:, None], torch.zeros_like(q), q)
        codes[:, i * group:(i + 1) * group] = q.clamp(-8, 7).long()
    return codes, scales


def codes_by_place(codes, R, C):
    """The stored codes, read place by place by the header's formula."""
    words = codes.cpu().numpy().view(np.uint32)
    G, S = words.shape[:2]
    out = np.zeros((16 * G, 128 * S), dtype=np.int64)
    flat = words.reshape(-1).astype(np.int64)
    r, c = np.meshgrid(np.arange(16 * G), np.arange(128 * S), indexing="ij")
    g, rr, s, w, j, i = r // 16, r % 16, c // 128, c % 128 // 32, c % 32 // 8, c % 8
    out = (flat[((g * S + s) * 64 + 16 * j + rr) * 4 + w] >> (4 * (i // 2) + 16 * (i % 2))) & 15
    assert (out[R:] == 8).all() and (out[:, C:] == 8).all()   # code 0 past the matrix
    return torch.from_numpy(out[:R, :C] - 8)


def scales_by_row(scales, R):
    s = scales.cpu()
    assert (s.transpose(1, 2).reshape(-1, s.shape[1])[R:] == 0).all()
    return s.transpose(1, 2).reshape(-1, s.shape[1])[:R]


def rows_of_blocked(v, R):
    """(G, S, 16, 32) -> (R, 32 S)."""
    return v.transpose(1, 2).reshape(16 * v.shape[0], -1)[:R]


def same(a, b):
    """Equal entry by entry, NaN with NaN."""
    a, b = a.double(), b.double()
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


SHAPES = [(1, 1), (16, 128), (17, 33), (3, 129), (40, 1000), (5, 257), (64, 96), (33, 8)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("group", nm.GROUPS)
@pytest.mark.parametrize("dtype,sdtype", [(torch.bfloat16, None), (torch.float16, None),
                                          (torch.float32, None),
                                          (torch.float32, torch.float16),
                                          (torch.float16, torch.bfloat16)])
def test_quantize_rows(R, C, group, dtype, sdtype):
    w = weights(R, C, dtype)
    codes, scales = nm.quantize(w.cuda(), group, scale_dtype=sdtype)
    q, s = plain_quantize(w, group, scales.dtype)
    assert torch.equal(codes_by_place(codes, R, C), q)
    assert torch.equal(scales_by_row(scales, R), s)
    back = nm.dequantize(codes, scales, C, group, rows=R).cpu()
    want = (q.double() * s.double().repeat_interleave(group, 1)[:, :C]).to(scales.dtype)
    assert torch.equal(back, want)


@pytest.mark.parametrize("R,K", [(16, 64), (33, 192), (7, 256), (48, 320)])
@pytest.mark.parametrize("group", nm.GROUPS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantize_compressed(R, K, group, dtype):
    w = weights(R, K, dtype)
    values, meta = nm.compress(w.cuda(), 2, 4, layout="blocked")
    codes, scales = nm.quantize(values, group, layout="blocked", rows=R)
    kept = rows_of_blocked(values.cpu(), R)
    q, s = plain_quantize(kept, group, scales.dtype)
    assert torch.equal(codes_by_place(codes, R, K // 2), q)
    assert torch.equal(scales_by_row(scales, R), s)
    back = nm.dequantize(codes, scales, K // 2, group, layout="blocked", rows=R)
    want = (q.double() * s.double().repeat_interleave(group, 1)[:, :K // 2]).to(scales.dtype)
    assert torch.equal(rows_of_blocked(back.cpu(), R), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_zeros_extremes_and_no_numbers(dtype):
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps   # the least number
    w = torch.zeros(6, 64, dtype=dtype)
    w[1, :32] = tiny                       # its scale rounds to zero, or to the least number
    w[2, 3] = torch.finfo(dtype).max
    w[2, 4] = -torch.finfo(dtype).max
    w[3, 5] = float("inf")
    w[3, 6] = 1.0
    w[4, 40] = float("nan")
    w[5] = -0.0
    codes, scales = nm.quantize(w.cuda(), 32)
    q, s = plain_quantize(w, 32, dtype)
    assert torch.equal(codes_by_place(codes, 6, 64), q)
    assert same(scales_by_row(scales, 6), s)
    back = nm.dequantize(codes, scales, 64, 32, rows=6).cpu()
    want = (q.double() * s.double().repeat_interleave(32, 1)).to(dtype)
    assert same(back, want)


def check_product(y, q, s, x, group, at=None):
    """y against the 64-bit product of codes q, scales s (R, groups) and x (K, T); at: the stored
    columns' places in x (R, C), for 2:4."""
    R, C = q.shape
    sr = s.double().repeat_interleave(group, 1)[:, :C]
    xd = x.double()
    w = q.double() * sr
    if at is not None:
        w = torch.zeros(R, x.shape[0], dtype=torch.float64).scatter_(1, at, w)
    want = w @ xd
    tol = ROUND[y.dtype] * want.abs() + 2 * (C + 2) * 2.0 ** -24 * (w.abs() @ xd.abs()) + 1e-30
    if y.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    assert (((y.double() - want).abs() <= tol)).all(), float(((y.double() - want).abs() / tol).max())


@pytest.mark.parametrize("R,K", [(1, 1), (16, 128), (17, 33), (40, 1000), (5, 7), (64, 2176),
                                 (100, 130)])
@pytest.mark.parametrize("T", [1, 2, 7, 16, 17, 32, 33, 70])
@pytest.mark.parametrize("group,dtype", [(32, torch.bfloat16), (64, torch.float16),
                                         (128, torch.bfloat16)])
def test_matvec_dense(R, K, T, group, dtype):
    w, x = weights(R, K, dtype), weights(K, T, torch.float64, 5).mul(50).to(dtype)
    codes, scales = nm.quantize(w.cuda(), group)
    q, s = plain_quantize(w, group, dtype)
    for out_dtype in (dtype, torch.float32):
        y = nm.matvec(codes, scales, x.cuda(), group, rows=R, out_dtype=out_dtype)
        assert y.dtype == out_dtype and y.shape == (R, T)
        check_product(y.cpu(), q, s, x, group)


@pytest.mark.parametrize("R,K", [(16, 64), (33, 192), (7, 256), (48, 1088), (130, 2112)])
@pytest.mark.parametrize("T", [1, 3, 16, 20, 40])
@pytest.mark.parametrize("group,dtype", [(32, torch.float16), (64, torch.bfloat16),
                                         (128, torch.float16), (128, torch.bfloat16)])
def test_matvec_compressed(R, K, T, group, dtype):
    w, x = weights(R, K, dtype), weights(K, T, torch.float64, 5).mul(50).to(dtype)
    values, meta = nm.compress(w.cuda(), 2, 4, layout="blocked")
    codes, scales = nm.quantize(values, group, layout="blocked", rows=R)
    keep = nm.mask(w.cuda(), 2, 4).cpu()
    at = keep.nonzero()[:, 1].view(R, K // 2)
    q, s = plain_quantize(w.gather(1, at), group, dtype)
    for out_dtype in (dtype, torch.float32):
        y = nm.matvec(codes, scales, x.cuda(), group, rows=R, meta=meta, out_dtype=out_dtype)
        check_product(y.cpu(), q, s, x, group, at)


@pytest.mark.parametrize("R,K,T,sparse", [(40, 40001, 1, False), (40, 21001, 5, False),
                                          (17, 30000, 8, False), (40, 24576, 3, True),
                                          (4200, 2048, 8, True), (9000, 5000, 3, False)])
def test_matvec_few_columns_of_long_or_many_rows(R, K, T, sparse):
    """Few columns that are too long to be held whole, or held whole by too many rows' workgroups."""
    dtype, group = torch.bfloat16, 64
    w, x = weights(R, K, dtype), weights(K, T, torch.float64, 5).mul(50).to(dtype)
    at = meta = None
    if sparse:
        at = nm.mask(w.cuda(), 2, 4).cpu().nonzero()[:, 1].view(R, K // 2)
        values, meta = nm.compress(w.cuda(), 2, 4, layout="blocked")
        codes, scales = nm.quantize(values, group, layout="blocked", rows=R)
    else:
        codes, scales = nm.quantize(w.cuda(), group)
    y = nm.matvec(codes, scales, x.cuda(), group, rows=R, meta=meta, out_dtype=torch.float32).cpu()
    some = torch.arange(0, R, max(1, R // 40))  # whole rows, every few
    rows = w[some]
    q, s = plain_quantize(rows if at is None else rows.gather(1, at[some]), group, dtype)
    check_product(y[some], q, s, x, group, None if at is None else at[some])


def test_matvec_agrees_with_the_products_it_stands_for():
    """The dequantised 2:4 pair through spmm, and the codes through matvec."""
    R, K, T = 64, 512, 8
    w, x = weights(R, K, torch.bfloat16).cuda(), weights(K, T, torch.bfloat16, 2).mul(50).cuda()
    values, meta = nm.compress(w, 2, 4, layout="blocked")
    codes, scales = nm.quantize(values, 64, layout="blocked", rows=R)
    back = nm.dequantize(codes, scales, K // 2, 64, layout="blocked", rows=R)
    a = nm.spmm(back, meta, x, 2, 4, out_dtype=torch.float32, layout="blocked", rows=R)
    b = nm.matvec(codes, scales, x, 64, rows=R, meta=meta, out_dtype=torch.float32)
    # spmm's weights are rounded to bfloat16 once, relative 2^-8 of each
    bound = 2.0 ** -7 * (nm.decompress(back, meta, 2, 4, K, "blocked", R).float().abs() @ x.float().abs())
    assert ((a - b).abs() <= bound + 1e-6).all()


def test_matvec_columns_do_not_mix():
    """Infinities and NaN in one column, or in a row block, reach only their own results."""
    R, K = 48, 256
    w = weights(R, K, torch.bfloat16).cuda()
    codes, scales = nm.quantize(w, 64)
    for T in (2, 5, 20):
        x = weights(K, T, torch.float64, 3).mul(50).to(torch.bfloat16).cuda()
        clean = nm.matvec(codes, scales, x, 64, rows=R)
        x[7, 1] = float("nan")
        y = nm.matvec(codes, scales, x, 64, rows=R)
        others = [t for t in range(T) if t != 1]
        assert torch.equal(y[:, others], clean[:, others])
        assert y[:, 1].isnan().all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 3, 16])
def test_matvec_infinities_and_the_largest_numbers(dtype, T):
    """Codes multiply as what they are: an infinity in X gives the infinities and NaN of the plain
    product, and numbers whose products with the codes are finite give finite sums."""
    R, K, group = 40, 256, 64
    gen = torch.Generator().manual_seed(5)
    q = torch.randint(-7, 8, (R, K), generator=gen)
    q[:, ::group] = 7  # every group's scale is 1
    q[0] = 0
    codes, scales = nm.quantize(q.to(dtype).cuda(), group)
    x = torch.zeros(K, T, dtype=dtype)
    x[5] = torch.finfo(dtype).max / 16
    y = nm.matvec(codes, scales, x.cuda(), group, rows=R, out_dtype=torch.float32).cpu()
    assert torch.equal(y.double(), q.double() @ x.double())
    x[5] = float("inf")
    y = nm.matvec(codes, scales, x.cuda(), group, rows=R, out_dtype=torch.float32).cpu()
    want = q.double()[:, 5:6] * torch.full((1, T), float("inf"), dtype=torch.float64)
    assert torch.equal(y.double().nan_to_num(1.0), want.nan_to_num(1.0))
    assert torch.equal(y.isnan(), want.isnan())


def test_matvec_is_repeatable_and_uses_the_current_stream():
    R, K, T = 1000, 4096, 5
    w = weights(R, K, torch.bfloat16).cuda()
    x = weights(K, T, torch.bfloat16, 3).cuda()
    codes, scales = nm.quantize(w, 64)
    first = nm.matvec(codes, scales, x, 64, rows=R)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x2 = x * 1
        again = nm.matvec(codes, scales, x2, 64, rows=R)
    side.synchronize()
    assert torch.equal(first, again)


def test_matvec_empty():
    codes, scales = nm.quantize(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), 64)
    y = nm.matvec(codes, scales, torch.zeros(64, 3, dtype=torch.bfloat16, device="cuda"), 64, rows=0)
    assert y.shape == (0, 3)
    codes, scales = nm.quantize(torch.zeros(5, 0, dtype=torch.bfloat16, device="cuda"), 64)
    y = nm.matvec(codes, scales, torch.zeros(0, 3, dtype=torch.bfloat16, device="cuda"), 64, rows=5)
    assert torch.equal(y.cpu(), torch.zeros(5, 3, dtype=torch.bfloat16))
