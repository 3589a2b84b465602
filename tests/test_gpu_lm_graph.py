"""The 4-bit, cross-entropy and orthogonalised-update calls captured into a graph: every replay,
on new inputs and with eager work between, gives the eager call's results bit for bit."""
import pytest
import torch

import masking_sparse_gemm_amd as nm

pytestmark = pytest.mark.gpu


def randn(*shape, seed, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


def case_quantize():
    def call(w):
        codes, scales = nm.quantize(w, 64)
        return codes, scales, nm.dequantize(codes, scales, w.shape[1], 64, rows=w.shape[0])
    return call, lambda seed: (randn(200, 1000, seed=seed),)


def case_matvec(R, K, T):
    codes, scales = nm.quantize(randn(R, K, seed=9), 64)
    return (lambda x: (nm.matvec(codes, scales, x, 64, rows=R),),
            lambda seed: (randn(K, T, seed=seed),))


def case_xent(V, K, T):
    def call(w, x, y, g):
        loss, lse = nm.xent(w, x, y)
        return (loss, lse, *nm.xent_grad(w, x, y, lse, g))

    def inputs(seed):
        gen = torch.Generator().manual_seed(seed)
        y = torch.randint(-1, V, (T,), generator=gen).cuda()
        return (randn(V, K, seed=seed) * 0.1, randn(K, T, seed=seed + 1), y,
                torch.rand(T, generator=gen).cuda())
    return call, inputs


def case_orthogonalize(R, K, dtype):
    return (lambda G: (nm.orthogonalize(G),), lambda seed: (randn(R, K, seed=seed, dtype=dtype),))


CASES = {
    "quantize": lambda: case_quantize(),
    "matvec one column": lambda: case_matvec(300, 1024, 1),
    "matvec few columns": lambda: case_matvec(300, 1024, 3),
    "matvec slices": lambda: case_matvec(64, 16384, 20),
    "xent": lambda: case_xent(3000, 200, 77),
    "xent large": lambda: case_xent(20000, 512, 300),
    "orthogonalize": lambda: case_orthogonalize(300, 500, torch.bfloat16),
    "orthogonalize fp32": lambda: case_orthogonalize(260, 130, torch.float32),
}


@pytest.mark.parametrize("name", CASES)
def test_replays(name):
    call, inputs = CASES[name]()
    state = inputs(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(*state)
    for replay in range(4):
        fresh = inputs(10 + replay)
        for old, new in zip(state, fresh):
            old.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, call(*fresh)):
            assert torch.equal(got, want)
        torch.cuda.synchronize()
