"""The 4-bit product held to the error that its sums can make, at long rows.

Codes enter the matrix cores as the 16-bit floats that they are, so products are exact.  A product
then passes at most 32 additions inside an instruction, group / 32 of an instruction's accumulator,
the scaled addition of its group's sum, one for each group of its row that the wave has, 16 of the
waves' sums and one for each slice of the row.  An addition is off by at most 2^-23 of its result
(an instruction's inner ones need not round to nearest), whatever is added, so with n the number
of these |d y| <= n 2^-23 sum |s q x| and, for a 16-bit result, its one rounding.
"""
import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests.test_gpu_quant import ROUND, plain_quantize, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nm.lib()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("R,K,T,group,sparse", [
    (40, 128, 1, 64, False), (33, 4096, 1, 128, False), (17, 32000, 1, 32, False),   # whole
    (40, 40001, 1, 64, False), (64, 40064, 1, 128, True),                            # slices
    (100, 4096, 2, 32, True), (19, 8192, 7, 64, False),                              # few columns
    (50, 11007, 5, 32, False), (130, 11008, 20, 64, True), (70, 4096, 32, 128, False),
    (5, 16384, 33, 64, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_sums_of_long_rows(R, K, T, group, sparse, dtype):
    w, x = weights(R, K, dtype), weights(K, T, torch.float64, 5).mul(50).to(dtype)
    at, meta, stored = None, None, w
    if sparse:
        at = nm.mask(w.cuda(), 2, 4).cpu().nonzero()[:, 1].view(R, K // 2)
        values, meta = nm.compress(w.cuda(), 2, 4, layout="blocked")
        codes, scales = nm.quantize(values, group, layout="blocked", rows=R)
        stored = w.gather(1, at)
    else:
        codes, scales = nm.quantize(w.cuda(), group)
    q, s = plain_quantize(stored, group, dtype)
    C = q.shape[1]
    v = q.double() * s.double().repeat_interleave(group, 1)[:, :C]
    if sparse:
        v = torch.zeros(R, K, dtype=torch.float64).scatter_(1, at, v)
    want, size = v @ x.double(), v.abs() @ x.double().abs()
    rows_of_slice = 64 * 1024 // 32 // (2 if T > 16 else 1)  # of X: 64 KB of 16 columns
    n = 32 + group // 32 + 1 + -(-C // group) + 16 + -(-K // rows_of_slice)
    for out in (torch.float32, dtype):
        y = nm.matvec(codes, scales, x.cuda(), group, rows=R, meta=meta, out_dtype=out).cpu()
        bound = n * 2.0 ** -23 * size
        if out == dtype:
            bound = bound + ROUND[dtype] * (want.abs() + bound)
            if dtype == torch.float16:
                bound = bound + 2.0 ** -25
        off = (y.double() - want).abs()
        assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("R,K,sparse", [(4700, 4096, True), (4700, 4096, False), (16400, 2048, True),
                                        (100, 7168, True), (200, 6144, False)])
def test_eight_columns_whole_and_in_slices(R, K, sparse):
    """Eight columns on both sides of the rule that parts them; some rows of each."""
    dtype, group = torch.bfloat16, 64
    w, x = weights(R, K, dtype), weights(K, 8, torch.float64, 5).mul(50).to(dtype)
    at, meta = None, None
    some = torch.arange(0, R, max(1, R // 40))
    if sparse:
        at = nm.mask(w.cuda(), 2, 4).cpu().nonzero()[:, 1].view(R, K // 2)
        values, meta = nm.compress(w.cuda(), 2, 4, layout="blocked")
        codes, scales = nm.quantize(values, group, layout="blocked", rows=R)
    else:
        codes, scales = nm.quantize(w.cuda(), group)
    y = nm.matvec(codes, scales, x.cuda(), group, rows=R, meta=meta, out_dtype=torch.float32).cpu()
    stored = w[some] if at is None else w[some].gather(1, at[some])
    q, s = plain_quantize(stored, group, dtype)
    C = q.shape[1]
    v = q.double() * s.double().repeat_interleave(group, 1)[:, :C]
    if sparse:
        v = torch.zeros(len(some), K, dtype=torch.float64).scatter_(1, at[some], v)
    n = 32 + group // 32 + 1 + -(-C // group) + 16 + -(-K // 2048)
    off = (y[some].double() - v @ x.double()).abs()
    assert (off <= n * 2.0 ** -23 * (v.abs() @ x.double().abs())).all()
