"""clip_grads at the ends of fp32: norms past its largest number and ratios below its smallest normal
one."""
import math

import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests.test_gpu_clip import check_clipped, check_norm, exact_norm, tensors

pytestmark = pytest.mark.gpu

# the largest entries here lie between 3.0e38 and 3.38e38, of which the first is below every type's largest
FEW, MANY = [(1000,), (70, 33)], [(40 + i,) for i in range(300)]


def huge(sizes, types, seed=0):
    return [((g.float().abs().clamp(max=1) * 0.1 + 0.9) * 3.3e38 * g.float().sign()).to(g.dtype)
            for g in tensors(sizes, types, seed=seed)]


@pytest.mark.parametrize("types", [(torch.float32,), (torch.bfloat16,), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("sizes", [FEW, MANY])
@pytest.mark.parametrize("most", [1.0, 1e-10, 3e-38, 1e38])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_norm_past_fp32(types, sizes, most, in_place):
    grads = huge(sizes, types)
    want = exact_norm(grads)
    assert want > 3.5e38
    keep = [g.clone() for g in grads]
    out = grads if in_place else [torch.full_like(g, 7.0) for g in grads]
    norm = nm.clip_grads(grads, most, out=None if in_place else out)
    assert float(norm) == math.inf and float(nm.grad_norm(keep)) == math.inf
    check_clipped(out, keep, want, float(torch.tensor(most)), norm)


@pytest.mark.parametrize("scale,most", [(1e30, 1e-10), (1e36, 0.5), (1e37, 1e-3), (1e20, 1e-30), (1e33, 1e-20)])
@pytest.mark.parametrize("types", [(torch.float32,), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("given", [False, True])
def test_a_ratio_below_the_smallest_normal_number(scale, most, types, given):
    grads = tensors(FEW, types, scale=scale)
    want = exact_norm(grads)
    most = float(torch.tensor(most))
    past = want > torch.finfo(torch.float32).max  # then a given norm is infinite, and clips nothing
    out = [torch.empty_like(g) for g in grads]
    norm = None
    if given:
        norm = torch.tensor(want, dtype=torch.float32, device="cuda")
    got = nm.clip_grads(grads, most, norm=norm, out=out)
    if past:
        assert float(got) == math.inf
    else:
        check_norm(got, want)
    check_clipped(out, grads, 0.0 if past and given else want, most, norm)


def test_an_infinity_among_huge_numbers_changes_nothing():
    grads = huge(FEW, (torch.float32,))
    grads[0][77] = -math.inf
    keep = [g.clone() for g in grads]
    assert float(nm.clip_grads(grads, 1.0)) == math.inf
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))


def test_a_given_norm_of_infinity_changes_nothing():
    grads = huge(FEW, (torch.float32,))
    keep = [g.clone() for g in grads]
    nm.clip_grads(grads, 1.0, norm=torch.tensor(math.inf, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
