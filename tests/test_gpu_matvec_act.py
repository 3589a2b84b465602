"""matvec_act against a 64-bit reference over what the codes stand for: one column and a few, the
joined slices, dense and 2:4 codes."""
import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests import act_ref as ref
from tests.test_gpu_spmm_act import DT

pytestmark = pytest.mark.gpu


def weights(R, K, dtype, group, sparse, seed):
    """(codes, scales, meta or None, the matrix in 64 bits): code * scale is exact there."""
    gen = torch.Generator().manual_seed(seed)
    w = (torch.randn(R, K, generator=gen) * K ** -0.5).to(DT[dtype]).cuda()
    meta = None
    if sparse:
        w, meta = nm.compress(w, 2, 4, layout="blocked")
        codes, scales = nm.quantize(w, group, layout="blocked", rows=R)
        C = K // 2
    else:
        codes, scales = nm.quantize(w, group)
        C = K
    word = codes.cpu().long() & 0xFFFFFFFF
    at = torch.tensor([4 * (i // 2) + 16 * (i % 2) for i in range(8)])
    q = ((word[..., None] >> at) & 15) - 8                       # G, S, lane, w, i
    G, S = q.shape[:2]
    q = q.view(G, S, 4, 16, 4, 8).permute(0, 3, 1, 4, 2, 5).reshape(16 * G, 128 * S)[:R, :C].double()
    s = scales.cpu().double().transpose(1, 2).reshape(16 * G, -1)[:R]
    dense = q * s.repeat_interleave(group, 1)[:, :C]
    if sparse:
        raw = meta.cpu().view(torch.uint8).view(G, K // 64, 16, 8).transpose(1, 2).reshape(16 * G, -1)[:R]
        place = ((raw[..., None] >> torch.tensor([0, 2, 4, 6])) & 3).reshape(R, C).long()
        full = torch.zeros(R, K, dtype=torch.float64)
        dense = full.scatter_(1, place + 4 * (torch.arange(C) // 2), dense)
    return codes, scales, meta, dense


def run(R, K, T, dtype, group, sparse, act, bias, residual, y=None, in_place=False, seed=0):
    codes, scales, meta, W = weights(R, K, dtype, group, sparse, seed)
    gen = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(K, T, generator=gen).to(DT[dtype])
    y_dt = DT[y or dtype]
    b = torch.randn(R, generator=gen) if bias else None
    r = torch.randn(R, T, generator=gen).to(y_dt) if residual else None
    cuda = lambda t: None if t is None else t.cuda()
    res = cuda(r)
    got = nm.matvec_act(codes, scales, x.cuda(), group, rows=R, meta=meta, bias=cuda(b), act=act,
                        residual=res, out_dtype=y_dt, out=res if in_place else None)
    sums = W @ x.double()
    want, bound, _, _ = ref.epilogue(sums, ref.sum_bound(2 * K, W.abs() @ x.double().abs()), b, act, r,
                                     y_dt)
    ref.check(got, want, bound, "Y")


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype,y", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32")])
def test_activations(act, dtype, y):
    run(200, 512, 1, dtype, 64, True, act, True, True, y)


@pytest.mark.parametrize("T", [1, 2, 5, 8, 17, 33])
@pytest.mark.parametrize("R,K,sparse,group", [(16, 64, True, 32), (33, 301, False, 32),
                                              (100, 1024, False, 128), (500, 4096, True, 64),
                                              (64, 16384, True, 128), (48, 20000, False, 64)])
def test_sizes(R, K, T, sparse, group):
    run(R, K, T, "bf16", group, sparse, "silu", True, True)


@pytest.mark.parametrize("bias,residual", [(0, 0), (1, 0), (0, 1)])
@pytest.mark.parametrize("T", [1, 3, 24])
def test_parts(bias, residual, T):
    run(130, 640, T, "fp16", 64, False, "gelu", bool(bias), bool(residual))


@pytest.mark.parametrize("T", [1, 4, 20])
def test_onto_the_residual_in_place(T):
    run(100, 16384, T, "bf16", 64, True, "none", False, True, in_place=True)


@pytest.mark.parametrize("T", [1, 5, 20])
def test_plain_call_is_matvec(T):
    codes, scales, meta, _ = weights(90, 1024, "bf16", 32, True, 4)
    x = torch.randn(1024, T).to(torch.bfloat16).cuda()
    assert torch.equal(nm.matvec_act(codes, scales, x, 32, rows=90, meta=meta),
                       nm.matvec(codes, scales, x, 32, rows=90, meta=meta))
