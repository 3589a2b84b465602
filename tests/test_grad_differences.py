"""spmm_act_grad against difference quotients of the activation in 64 bits, entry by entry: of X, of W and of
the bias, each moved on its own around the Z that the kernel is given.  On the CPU: the bound that the
kernel is held to does not let a gradient pass that lacks a term of its slope."""

import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests import act_ref as ref

R, K, T = 48, 64, 20
H = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def case(dtype):
    gen = torch.Generator().manual_seed(11)
    w = (torch.randn(R, K, generator=gen) / 6).to(TYPES[dtype])
    pruned = w.view(R, K // 4, 4)
    least = torch.argsort(pruned.float().abs(), dim=2, descending=False, stable=True)[..., :2]
    w = pruned.scatter(2, least, 0).view(R, K)
    x = torch.randn(K, T, generator=gen).to(TYPES[dtype])
    z = (torch.randn(R, T, generator=gen) * 2).to(TYPES[dtype])
    dy = torch.randn(R, T, generator=gen).to(TYPES[dtype])
    return w, x, z, dy


def quotients(w, x, z, dy, act):
    """{name: (quotient, what it may be off by)}.  The quotient is off by h^2 / 6 of a third derivative
    (below 4 in size for |z| < 10) times the move's cube, and by 64-bit rounding over h."""
    w, x, z, dy = (t.double() for t in (w, x, z, dy))
    if act.startswith("relu"):  # no kink within reach of a move
        assert float(z.abs().min()) > 10 * H * max(1.0, float(w.abs().max()), float(x.abs().max()))

    def slope_along(move):  # of act at z, moved by h move, over a last dimension of moves
        up, down = (ref.act(z[..., None] + s * H * move, act) for s in (1, -1))
        return (up - down) / (2 * H) * dy[..., None]

    each = lambda move: H ** 2 * move.abs() ** 3 * dy.abs()[..., None] + \
        4 * 2.0 ** -52 / H * (z.abs()[..., None] + 1) ** 2 * dy.abs()[..., None]
    by_x, by_w, one = w[:, None, :].expand(R, T, K), x.t()[None].expand(R, T, K), torch.ones(R, T, 1).double()
    return {"dX": (slope_along(by_x).sum(0).t(), each(by_x).sum(0).t()),
            "dW": (slope_along(by_w).sum(1), each(by_w).sum(1)),
            "dbias": (slope_along(one).sum((1, 2)), each(one).sum((1, 2)))}


def bounds(w, x, z, dy, act, dtype):
    return {k: b for k, (_, b) in ref.gradient(w, x, z, dy, act, TYPES[dtype]).items()}


def missing_term(z, act):
    """The slope without its second term."""
    if act == "silu":
        return torch.sigmoid(z)
    if act == "gelu":
        return torch.special.ndtr(z)
    return 0.5 * (1 + torch.tanh(ref.ROOT * (z + 0.044715 * z ** 3)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_a_gradient_that_lacks_a_term_is_past_the_bound(act, dtype):
    w, x, z, dy = case(dtype)
    q, b = quotients(w, x, z, dy, act), bounds(w, x, z, dy, act, dtype)
    dz = dy.double() * missing_term(z.double(), act)
    wrong = {"dX": w.double().t() @ dz, "dW": dz @ x.double().t(), "dbias": dz.sum(1)}
    right = dy.double() * ref.slope(z.double(), act)
    good = {"dX": w.double().t() @ right, "dW": right @ x.double().t(), "dbias": right.sum(1)}
    for name, (value, off) in q.items():
        assert bool(((good[name] - value).abs() <= off).all()), name
        past = (wrong[name] - value).abs() > b[name] + off
        assert float(past.double().mean()) > 0.9, name   # nearly every entry on its own


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ref.ACTS)
def test_kernel_against_differences(act, dtype):
    w, x, z, dy = case(dtype)
    values, meta = nm.compress(w.cuda(), 2, 4)
    assert torch.equal(nm.decompress(values, meta, 2, 4, K).cpu(), w)
    names = ("dX", "dW", "dbias")
    got = nm.spmm_act_grad(values, meta, x.cuda(), dy.cuda(), z.cuda(), act=act, want=names)
    q, b = quotients(w, x, z, dy, act), bounds(w, x, z, dy, act, dtype)
    for name, g in zip(names, got):
        ref.check(g, q[name][0], b[name] + q[name][1], name)
