"""grad_norm and clip_grads against 64-bit sums: mixed types, odd addresses and sizes, many tensors,
the ends of the types' ranges."""
import math

import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests import act_ref as ref

pytestmark = pytest.mark.gpu

TYPES = (torch.float32, torch.float16, torch.bfloat16)


def tensors(sizes, types=TYPES, scale=1.0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=gen) * scale).to(types[i % len(types)]).cuda()
            for i, s in enumerate(sizes)]


def exact_norm(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def check_norm(got, want):
    # groups of eight in fp32 (8 roundings), fp64 from there, one rounding
    assert got.dtype == torch.float32 and got.dim() == 0
    assert abs(float(got) - want) <= 6 * ref.F32 * want, (float(got), want)


def check_clipped(got, grads, want_norm, most, norm):
    f = most / want_norm if want_norm > most else 1.0
    for a, g in zip(got, grads):
        if f == 1.0:
            assert torch.equal(a, g)
            continue
        w = g.double() * f
        # the norm (6 roundings), the ratio and the product round once each, then the result
        off = 8 * ref.F32 * w.abs()
        ref.check(a, w, (off + ref.rounding(w, g.dtype)) * (1 + 2 * ref.HALF[g.dtype]), "clipped")


SIZES = {
    "one": [(1,)],
    "small": [(3,), (5, 7), (8192,), (8193,), (1, 1)],
    "empty among them": [(0,), (100,), (0, 5), (7,)],
    "many": [(17 + 31 * (i % 50),) for i in range(300)],
    "large": [(3000, 1001), (123457,), (2048, 2048)],
}


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("over", [0.5, 3.0])
def test_norm_and_clip(sizes, over):
    grads = tensors(SIZES[sizes])
    want = exact_norm(grads)
    check_norm(nm.grad_norm(grads), want)
    most = want / over
    out = [torch.full_like(g, 7.0) for g in grads]
    norm = nm.clip_grads(grads, most, out=out)
    check_norm(norm, want)
    check_clipped(out, grads, want, most, norm)
    before = [g.clone() for g in grads]
    again = nm.clip_grads(grads, most)
    assert torch.equal(again, norm)
    for a, b in zip(grads, out):
        assert torch.equal(a, b)
    assert all(a.shape == b.shape for a, b in zip(grads, before))


def test_same_result_every_time():
    grads = tensors([(1000, 1000), (333,)] * 40)
    first = nm.grad_norm(grads)
    for _ in range(3):
        assert torch.equal(nm.grad_norm(grads), first)


@pytest.mark.parametrize("dtype", TYPES)
def test_views_at_any_element_and_nothing_beside_them(dtype):
    flat = torch.randn(40000).to(dtype).cuda()
    keep = flat.clone()
    cuts = [(1, 130), (131, 8200), (8333, 31000), (31001, 39999)]
    views = [flat[a:b] for a, b in cuts]
    want = exact_norm(views)
    nm.clip_grads(views, want / 2)
    inside = torch.zeros(40000, dtype=torch.bool, device="cuda")
    for a, b in cuts:
        inside[a:b] = True
    assert torch.equal(flat[~inside], keep[~inside])
    check_clipped([flat[inside]], [keep[inside]], want, want / 2, None)


def test_transposed_matrices():
    g = torch.randn(300, 70).cuda()
    check_norm(nm.grad_norm([g.t()]), exact_norm([g]))
    with pytest.raises(ValueError):
        nm.grad_norm([g[:, :30]])


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e18, 3e37])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_squares_past_fp32(scale, dtype):
    grads = tensors([(1000,), (70,)], types=(dtype,), scale=scale)
    grads[0] = grads[0].clamp(-3e38, 3e38)
    want = exact_norm(grads)
    if want > 3.4e38:
        grads = [g / 64 for g in grads]
        want = exact_norm(grads)
    check_norm(nm.grad_norm(grads), want)
    out = [torch.empty_like(g) for g in grads]
    nm.clip_grads(grads, want / 4, out=out)
    check_clipped(out, grads, want, want / 4, None)


def test_mixed_magnitudes():
    """Eight neighbours of which one square fits fp32 and seven underflow it, and the reverse."""
    a = torch.full((4096,), 1e-25)
    a[::8] = 1.0
    b = torch.full((4096,), 1e-3)
    b[5] = 1e30
    for t in (a, b, torch.cat([a, b]), torch.zeros(100)):
        check_norm(nm.grad_norm([t.cuda()]), exact_norm([t]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_rows_of_zeros(dtype):
    """A gradient of an embedding: few rows in use; zeros of either sign, and a subnormal among them."""
    g = torch.zeros(300, 128, dtype=dtype)
    g[::2] = -0.0
    tiny = torch.finfo(dtype).smallest_normal / 2
    g[7, 5] = tiny
    check_norm(nm.grad_norm([g.cuda()]), exact_norm([g]))
    g[41] = torch.randn(128)
    check_norm(nm.grad_norm([g.cuda()]), exact_norm([g]))


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_no_number_changes_nothing(bad):
    grads = tensors([(1000,), (50,)])
    grads[1][3] = bad
    keep = [g.clone() for g in grads]
    norm = nm.clip_grads(grads, 1.0)
    assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
    for a, b in zip(grads, keep):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_zeros_and_a_limit_of_zero():
    z = [torch.zeros(100, device="cuda")]
    assert float(nm.clip_grads(z, 0.0)) == 0 and bool((z[0] == 0).all())
    g = tensors([(100,), (9,)])
    nm.clip_grads(g, 0.0)
    assert all(bool((t == 0).all()) for t in g)


def test_a_given_norm():
    grads = tensors([(1000,), (77,)])
    want = exact_norm(grads)
    given = torch.tensor(2 * want, device="cuda", dtype=torch.float32)
    out = [torch.empty_like(g) for g in grads]
    got = nm.clip_grads(grads, want, norm=given, out=out)  # as of two ranks
    assert got is given
    check_clipped(out, grads, float(given), want, None)


def test_the_same_tensor_twice():
    g = torch.randn(1000, device="cuda")
    check_norm(nm.grad_norm([g, g]), exact_norm([g, g]))
    with pytest.raises(nm.NMError) as e:
        nm.clip_grads([g, g], 1.0)
    assert nm.STATUS[e.value.status] == "alias"
    with pytest.raises(nm.NMError):
        nm.clip_grads([g[:600], g[400:]], 1.0)
    out = [torch.empty_like(g), torch.empty_like(g)]
    nm.clip_grads([g, g], 1.0, out=out)
    assert torch.equal(out[0], out[1])


def test_lists_and_single_tensors():
    g = torch.randn(50, 3, 2, device="cuda")
    assert torch.equal(nm.grad_norm(g), nm.grad_norm([g]))
    with pytest.raises(ValueError):
        nm.grad_norm([])
    with pytest.raises(ValueError):
        nm.clip_grads([g], 1.0, out=[g[:10]])
    with pytest.raises(nm.NMError):
        nm.clip_grads([g], -1.0)
    with pytest.raises(nm.NMError):
        nm.clip_grads([g], math.nan)
