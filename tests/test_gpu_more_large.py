"""Results past 2^31 entries of the epilogue, its gradient, clipping and logits calls, checked on samples
of rows and columns against the 64-bit forms (inputs are small blocks repeated on the GPU)."""
import math

import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests import act_ref as ref
from tests.test_gpu_logits import expected

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
R, K, T = 70_000, 64, 32_768
ROWS = [0, 1, 255, 999, 32_767, 65_535, 65_536, R - 257, R - 1]
COLS = [0, 7, 4095, 4096, 30_001, T - 1]
assert R * T > 2 ** 31


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF)


@pytest.fixture(autouse=True)
def empty():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def weight():
    values, meta = nm.compress(randn(R, K, seed=1).cuda(), 2, 4, layout="blocked")
    return values, meta, nm.decompress(values, meta, 2, 4, K, layout="blocked", rows=R).cpu()


def test_product_with_its_epilogue(weight):
    values, meta, W = weight
    X, r, b = randn(K, T, seed=2), randn(1000, T, seed=3), torch.randn(R)
    Y, Z = nm.spmm_act(values, meta, X.cuda(), bias=b.cuda(), act="silu", residual=r.cuda().repeat(70, 1),
                       keep=True, layout="blocked", rows=R)
    w, x = W[ROWS].double(), X.double()
    off = ref.sum_bound(K // 2, w.abs() @ x.abs())
    wy, by, wz, bz = ref.epilogue(w @ x, off, b[ROWS], "silu", r[[i % 1000 for i in ROWS]], BF, BF)
    ref.check(Y[ROWS], wy, by, "Y")
    ref.check(Z[ROWS], wz, bz, "Z")


def test_gradient(weight):
    values, meta, W = weight
    X, z, dy = randn(K, T, seed=4), randn(1000, T, seed=5), randn(1000, T, seed=6)
    dW, dX, db, dZ = nm.spmm_act_grad(values, meta, X.cuda(), dy.cuda().repeat(70, 1),
                                      z.cuda().repeat(70, 1), act="gelu", layout="blocked", rows=R,
                                      want=("dW", "dX", "dbias", "dZ"))
    at = [i % 1000 for i in ROWS]
    rows = ref.gradient(None, X, z[at], dy[at], "gelu", BF)
    ref.check(dZ[ROWS], *rows["dZ"], "dZ")
    ref.check(db[ROWS], *rows["dbias"], "dbias")
    ref.check(dW[ROWS], *rows["dW"], "dW")
    cols = ref.gradient(W, None, z[:, COLS].repeat(70, 1), dy[:, COLS].repeat(70, 1), "gelu", BF)
    ref.check(dX[:, COLS], *cols["dX"], "dX")


def test_clipping():
    base = randn(1 << 20, seed=7)
    grad = base.cuda().repeat(2049)
    assert grad.numel() > 2 ** 31
    want = math.sqrt(2049 * float(base.double().square().sum()))
    norm = nm.clip_grads([grad], want / 4)
    assert abs(float(norm) - want) <= 6 * ref.F32 * want
    w = base.double() / 4
    off = (8 * ref.F32 * w.abs() + ref.rounding(w, BF)) * (1 + 2 * ref.HALF[BF])
    for i in (0, 1, 1023, 2047, 2048):
        ref.check(grad[i << 20:(i + 1) << 20], w, off, f"block {i}")


@pytest.mark.parametrize("each", [20, 3000])
def test_logits(each):
    """Few tokens are counted in LDS, many through a table."""
    V, columns = 131_072, 16_500
    assert V * columns > 2 ** 31
    assert (nm.lib().nm_adjust_logits_workspace_bytes(V, columns, each * columns) > 0) == (each > 1000)
    base = randn(V, 33, seed=8)
    gen = torch.Generator().manual_seed(9)
    tokens = torch.randint(V - 5000, V, (each * columns,), generator=gen)
    starts = torch.arange(columns + 1) * each
    rep, freq = torch.rand(columns, generator=gen) + 1, torch.rand(columns, generator=gen) * 0.1
    x = base.cuda().repeat(1, 500)
    out = nm.adjust_logits(x, tokens.cuda(), starts.cuda(), repetition=rep.cuda(), frequency=freq.cuda(), out=x)
    at = torch.tensor([0, 1, 31, 32, 8191, 16_383, 16_384, columns - 1])
    own = torch.cat([tokens[t * each:(t + 1) * each] for t in at.tolist()])
    ref.check(out[:, at.cuda()], *expected(base[:, at % 33], own, torch.arange(len(at) + 1) * each, None, rep[at],
                                           None, freq[at], None, None), "logits")
