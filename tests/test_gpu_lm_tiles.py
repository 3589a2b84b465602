"""Every tile of the dense product, in the cross entropy, its gradient and the orthogonalised update,
with ragged ends, pieces of the vocabulary and split sums, against the 64-bit forms (on the GPU).

The sizes and the tiles they take are those of lm_sizes.py.  Tolerances: test_gpu_xent's derivation,
element by element, and test_gpu_orth's bounds.
"""
import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests import test_gpu_orth as orth
from tests.lm_sizes import ORTH, XENT
from tests.test_gpu_xent import ROUND, plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nm.lib()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def within(got, want, bound, name):
    off = (got.double() - want).abs()
    assert (off <= bound).all(), (name, float((off / bound).max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V,K,T", XENT)
def test_cross_entropy(V, K, T, dtype):
    gen = torch.Generator("cuda").manual_seed(V + 31 * K + 977 * T)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    W, X = (randn(V, K) / K ** 0.5).to(dtype), randn(K, T).to(dtype)
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    y[1], y[2], y[T - 1] = -100, V, V - 1
    gout = torch.rand(T, generator=gen, device="cuda") * 64 / T  # dW within fp16's normal numbers
    loss, lse = nm.xent(W, X, y)
    dW, dX = nm.xent_grad(W, X, y, lse, gout)
    with torch.device("cuda"):
        want = plain(W, X, y, gout)
    left = ~want["live"]
    tol = (2 * want["dl"] + (V / 32 + 64) * 2.0 ** -24
           + 2.0 ** -21 * (1 + want["l"].abs().amax(0)))
    within(lse, want["lse"], tol, "lse")
    within(loss, want["loss"], 2 * tol, "loss")
    assert (loss[left] == 0).all() and (dX[:, left] == 0).all()
    u = ROUND[dtype]
    e = float(2 * tol.max()) + (max(V, T) + 64) * 2.0 ** -24
    small = 2.0 ** -37 * float(want["gmax"]) if dtype == torch.float16 else 0.0
    tiny = 2.0 ** -25 if dtype == torch.float16 else 1e-30
    for got, name, mag, n in ((dW, "dW", "mW", X.double().abs().sum(1)[None]),
                              (dX, "dX", "mX", W.double().abs().sum(0)[:, None])):
        within(got, want[name],
               (u + e) * want[mag] * (1 + u) + u * want[name].abs() + small * n + tiny, name)


@pytest.mark.parametrize("R,K,dtype", ORTH)
def test_orthogonalize(R, K, dtype):
    gen = torch.Generator("cuda").manual_seed(R * 7919 + K)
    G = (torch.randn(R, K, generator=gen, device="cuda") * 0.25).to(dtype)
    got = nm.orthogonalize(G)
    want = orth.plain(G)
    assert float((got.double() - want).norm() / want.norm()) <= orth.BOUND[dtype]
    # no tile, and no 32 x 32 part of one, is off on its own: entries are rounded alike, so a part's
    # difference is the whole's but for its share of chance
    tall, wide = -(-R // 32) * 32, -(-K // 32) * 32
    off = torch.zeros(tall, wide, dtype=torch.float64, device="cuda")
    off[:R, :K] = (got.double() - want) ** 2
    parts = off.view(tall // 32, 32, wide // 32, 32).sum((1, 3))
    mean = float(want.square().mean()) * 1024
    assert float(parts.max()) <= (3 * orth.BOUND[dtype]) ** 2 * mean
