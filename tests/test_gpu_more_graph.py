"""The epilogue, gradient, clipping and logits calls captured into graphs: every replay, on new inputs
and with eager work between, gives the eager call's results bit for bit; and a training and a
serving step of them together."""
import math

import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests import act_ref as ref
from tests.test_gpu_lm_graph import randn

pytestmark = pytest.mark.gpu


def pair(R, K, seed=9):
    return nm.compress(randn(R, K, seed=seed) * K ** -0.5, 2, 4, layout="blocked")


def case_spmm_act(R, K, T):
    values, meta = pair(R, K)
    bias = torch.randn(R, device="cuda")

    def call(x, r):
        return nm.spmm_act(values, meta, x, bias=bias, act="silu", residual=r, keep=True,
                           layout="blocked", rows=R)
    return call, lambda seed: (randn(K, T, seed=seed), randn(R, T, seed=seed + 1))


def case_grad(R, K, T):
    values, meta = pair(R, K)

    def call(x, z, dy):
        return nm.spmm_act_grad(values, meta, x, dy, z, act="gelu", layout="blocked", rows=R,
                                want=nm.GRADS)
    return call, lambda seed: (randn(K, T, seed=seed), randn(R, T, seed=seed + 1),
                               randn(R, T, seed=seed + 2))


def case_matvec_act(R, K, T):
    codes, scales = nm.quantize(randn(R, K, seed=9), 64)
    return (lambda x, r: (nm.matvec_act(codes, scales, x, 64, rows=R, act="gelu", residual=r),),
            lambda seed: (randn(K, T, seed=seed), randn(R, T, seed=seed + 1)))


def case_clip(count):
    def call(*grads):
        out = [torch.empty_like(g) for g in grads]
        return (nm.clip_grads(grads, 1.0, out=out), nm.grad_norm(grads), *out)
    return call, lambda seed: tuple(randn(50 + 13 * i, 40, seed=seed + i) for i in range(count))


def case_logits(V, T, count):
    starts = (torch.arange(T + 1) * (count // T)).cuda()

    def inputs(seed):
        gen = torch.Generator().manual_seed(seed)
        return (randn(V, T, seed=seed), torch.randint(0, V, (count,), generator=gen).cuda(),
                (torch.rand(T, generator=gen) + 1).cuda())

    def call(x, tokens, rep):
        return (nm.adjust_logits(x, tokens, starts, repetition=rep, frequency=rep),)
    return call, inputs


CASES = {
    "spmm_act": lambda: case_spmm_act(300, 512, 136),
    "spmm_act ragged": lambda: case_spmm_act(300, 512, 61),
    "spmm_act one token": lambda: case_spmm_act(300, 512, 1),
    "grad": lambda: case_grad(256, 512, 128),
    "grad ragged, split": lambda: case_grad(2001, 64, 77),
    "matvec_act": lambda: case_matvec_act(300, 1024, 1),
    "matvec_act slices": lambda: case_matvec_act(64, 16384, 20),
    "clip": lambda: case_clip(5),
    "clip many": lambda: case_clip(130),
    "logits": lambda: case_logits(5000, 6, 600),
    "logits through the table": lambda: case_logits(3000, 2, 4_000_000),
}


def capture(call, state):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(*state)
    return graph, out


@pytest.mark.parametrize("name", CASES)
def test_replays(name):
    call, inputs = CASES[name]()
    state = inputs(1)
    graph, out = capture(call, state)
    for replay in range(4):
        fresh = inputs(10 + replay)
        for old, new in zip(state, fresh):
            old.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, call(*fresh)):
            assert torch.equal(got, want)
        torch.cuda.synchronize()


def test_two_graphs_in_turn():
    """Two captured calls with workspaces of their own, replayed in turn and on two streams."""
    call, inputs = case_grad(257, 512, 77)
    states = [inputs(1), inputs(2)]
    graphs = [capture(call, s) for s in states]
    want = [[t.clone() for t in call(*s)] for s in states]
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for s, (g, _) in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))


def test_a_training_step_together():
    """Two layers, x2 = x1 + W2 silu(W1 x1 + b1): the gradients against 64 bits through the stored
    tensors, clipped together."""
    D, H, T = 128, 320, 45
    w1, w2 = randn(H, D, seed=1) * D ** -0.5, randn(D, H, seed=2) * H ** -0.5
    b1 = torch.randn(H, device="cuda") * 0.1
    x1 = randn(D, T, seed=3)
    pairs = [nm.compress(w, 2, 4, layout="blocked") for w in (w1, w2)]
    dense = [nm.decompress(*p, 2, 4, w.shape[1], layout="blocked", rows=w.shape[0]).cpu()
             for p, w in zip(pairs, (w1, w2))]
    h, z = nm.spmm_act(*pairs[0], x1, bias=b1, act="silu", keep=True, layout="blocked", rows=H)
    x2 = nm.spmm_act(*pairs[1], h, residual=x1, layout="blocked", rows=D)
    W1, W2, X1 = dense[0].double(), dense[1].double(), x1.cpu().double()
    off = ref.sum_bound(D // 2, W1.abs() @ X1.abs())
    ref.check(h, *ref.epilogue(W1 @ X1, off, b1.cpu(), "silu", None, torch.bfloat16)[:2], "h")
    Hs = h.cpu().double()
    off = ref.sum_bound(H // 2, W2.abs() @ Hs.abs())
    ref.check(x2, *ref.epilogue(W2 @ Hs, off, None, "none", x1.cpu(), torch.bfloat16)[:2], "x2")
    dx2 = randn(D, T, seed=4)
    g2, dh = nm.spmm_act_grad(*pairs[1], h, dx2, layout="blocked", rows=D, want=("dW", "dX"))
    g1, dx1, db = nm.spmm_act_grad(*pairs[0], x1, dh, z, act="silu", layout="blocked", rows=H)
    want2 = ref.gradient(dense[1], h.cpu(), None, dx2.cpu(), "none", torch.bfloat16)
    ref.check(g2, *want2["dW"], "g2")
    ref.check(dh, *want2["dX"], "dh")
    want1 = ref.gradient(dense[0], x1.cpu(), z.cpu(), dh.cpu(), "silu", torch.bfloat16)
    for got, name in ((g1, "dW"), (dx1, "dX"), (db, "dbias")):
        ref.check(got, *want1[name], name)
    grads = [g1, g2, db]
    before = [g.clone() for g in grads]
    total = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    norm = nm.clip_grads(grads, total / 3)
    assert abs(float(norm) - total) <= 6 * ref.F32 * total
    for g, b in zip(grads, before):
        w = b.double() / 3
        ref.check(g, w, (8 * ref.F32 * w.abs() + ref.rounding(w, g.dtype)) * (1 + 2 * ref.HALF[g.dtype]),
                  "clipped")


def test_a_serving_step_together():
    """One token through a 4-bit 2:4 layer onto its residual and the head, then its penalties: each
    stage against 64 bits from what the stage before stored."""
    from tests.test_gpu_logits import expected
    from tests.test_gpu_matvec_act import weights

    D, V = 256, 1000
    codes, scales, meta, W = weights(D, D, "bf16", 64, True, 1)
    hc, hs, _, Wh = weights(V, D, "bf16", 64, False, 2)
    x = randn(D, 1, seed=3)
    start = x.clone()
    nm.matvec_act(codes, scales, x, 64, rows=D, meta=meta, act="gelu", out=(y := torch.empty_like(x)))
    stream = nm.matvec_act(codes, scales, y, 64, rows=D, meta=meta, residual=x, out=x)
    logits = nm.matvec_act(hc, hs, stream, 64, rows=V, out_dtype=torch.float32)
    tokens, starts = torch.tensor([5, 7, 5]).cuda(), torch.tensor([0, 3]).cuda()
    rep = torch.tensor([1.3]).cuda()
    final = nm.adjust_logits(logits, tokens, starts, repetition=rep)
    bound = lambda M, v: ref.sum_bound(2 * D, M.abs() @ v.abs())
    yd, sd = y.cpu().double(), stream.cpu().double()
    ref.check(y, *ref.epilogue(W @ start.cpu().double(), bound(W, start.cpu().double()), None, "gelu", None,
                               torch.bfloat16)[:2], "y")
    ref.check(stream, *ref.epilogue(W @ yd, bound(W, yd), None, "none", start.cpu(),
                                    torch.bfloat16)[:2], "stream")
    ref.check(logits, *ref.epilogue(Wh @ sd, bound(Wh, sd), None, "none", None, torch.float32)[:2], "logits")
    ref.check(final, *expected(logits.cpu(), tokens.cpu(), starts.cpu(), None, rep.cpu(), None, None,
                               None, None), "final")
