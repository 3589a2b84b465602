"""The orthogonalised update against the same steps in 64 bits.

Tolerances are on the Frobenius norm of the difference over the result's.  fp16 operands carry
2^-12 relative an entry; a CPU model of the same roundings (X in fp32, operands in fp16) on
spectra flat and steep puts the result within 3.4e-3 with bfloat16's own output rounding (1.7e-3)
included, and with two-part operands within 3e-5: the bounds are 1.5 times those, plus fp16's
output rounding (2.1e-4) where it applies.
"""
import pytest
import torch

import masking_sparse_gemm_amd as nm

pytestmark = pytest.mark.gpu

BOUND = {torch.bfloat16: 5e-3, torch.float16: 3.6e-4, torch.float32: 4.5e-5}
COEFS = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nm.lib()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def plain(G, steps=5, eps=1e-7):
    X = G.double()
    X = X / (X.square().sum().sqrt() + eps)
    tall = X.shape[0] > X.shape[1]
    X = X.t() if tall else X
    a, b, c = COEFS
    for _ in range(steps):
        A = X @ X.t()
        X = a * X + (b * A + c * A @ A) @ X
    return X.t() if tall else X


def update(R, K, dtype, seed=0, steep=False):
    g = torch.Generator().manual_seed(R * 7919 + K + seed)
    G = torch.randn(R, K, generator=g, dtype=torch.float64) * 1e-3
    if steep:
        n = min(R, K)
        s = torch.arange(1, n + 1, dtype=torch.float64) ** -1.0
        G = (torch.randn(R, n, generator=g, dtype=torch.float64) * s) @ \
            torch.randn(n, K, generator=g, dtype=torch.float64) * 1e-3
    return G.to(dtype)


def off(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("R,K", [(1, 1), (1, 50), (50, 1), (3, 5), (64, 64), (65, 63), (63, 129),
                                 (130, 100), (200, 333), (512, 256), (257, 640)])
def test_small_and_odd_sizes(R, K, dtype):
    G = update(R, K, dtype)
    assert off(nm.orthogonalize(G.cuda()), plain(G)) <= BOUND[dtype]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,K", [(1500, 1600), (3000, 1500), (1024, 4100)])
def test_larger_tiles(R, K, dtype):
    G = update(R, K, dtype)
    want = plain(G.cuda()).cpu()
    assert off(nm.orthogonalize(G.cuda()), want) <= BOUND[dtype]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_steep_spectrum(dtype):
    for R, K in ((300, 500), (500, 300)):
        G = update(R, K, dtype, steep=True)
        assert off(nm.orthogonalize(G.cuda()), plain(G)) <= BOUND[dtype]


def test_singular_values_end_near_one():
    G = update(256, 384, torch.float32)
    s = torch.linalg.svdvals(nm.orthogonalize(G.cuda()).cpu().double())
    assert s.min() > 0.6 and s.max() < 1.3


@pytest.mark.parametrize("steps", [1, 2, 6])
def test_steps(steps):
    G = update(100, 200, torch.float32)
    assert off(nm.orthogonalize(G.cuda(), steps=steps), plain(G, steps)) <= BOUND[torch.float32]


@pytest.mark.parametrize("dtype,scale", [(torch.bfloat16, 2.0 ** 120), (torch.bfloat16, 2.0 ** -110),
                                         (torch.float32, 2.0 ** 100), (torch.float32, 2.0 ** -100),
                                         (torch.float16, 2.0 ** 20), (torch.float16, 2.0 ** -6)])
def test_any_size_of_update(dtype, scale):
    """The norm neither overflows nor vanishes; eps = 0 leaves the update's size without effect."""
    G = (update(96, 160, torch.float64) * scale).to(dtype)
    assert off(nm.orthogonalize(G.cuda(), eps=0.0), plain(G, eps=0.0)) <= BOUND[dtype]


def test_eps_holds_small_updates_back():
    G = update(64, 96, torch.float32) * 1e-7   # norm about 8e-9
    assert off(nm.orthogonalize(G.cuda(), eps=1e-7), plain(G, eps=1e-7)) <= BOUND[torch.float32]


def test_zero_and_not_finite():
    Z = torch.zeros(70, 90, dtype=torch.bfloat16, device="cuda")
    assert (nm.orthogonalize(Z) == 0).all()
    Z[3, 4] = float("nan")
    assert nm.orthogonalize(Z).isnan().any()
    Z[3, 4] = float("inf")
    assert nm.orthogonalize(Z).isnan().any()


def test_in_place_repeatable_and_on_the_current_stream():
    G = update(300, 200, torch.bfloat16).cuda()
    first = nm.orthogonalize(G)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        H = G * 1
        again = nm.orthogonalize(H, out=H)
    side.synchronize()
    assert again is H and torch.equal(first, H)


def test_empty():
    for shape in ((0, 5), (5, 0)):
        assert nm.orthogonalize(torch.zeros(shape, dtype=torch.bfloat16, device="cuda")).shape == shape
