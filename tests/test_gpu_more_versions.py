"""Tensors that the epilogue, clipping and logits calls write in place have moved version counters, so that a
backward pass which saved one of them says so instead of giving a wrong gradient."""
import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests.test_gpu_lm_graph import randn

pytestmark = pytest.mark.gpu


def pair():
    return nm.compress(randn(64, 64, seed=1), 2, 4, layout="blocked")


def codes():
    return nm.quantize(randn(64, 64, seed=1), 64)


CALLS = {
    "spmm_act": lambda t: nm.spmm_act(*pair(), randn(64, 8, seed=2), residual=t, out=t, layout="blocked", rows=64),
    "matvec_act": lambda t: nm.matvec_act(*codes(), randn(64, 8, seed=2), 64, rows=64, residual=t, out=t),
    "clip_grads": lambda t: nm.clip_grads([randn(5, 5, seed=3), t], 1e-3),
    "clip_grads out": lambda t: nm.clip_grads([randn(64, 8, seed=3)], 1e-3, out=[t]),
    "adjust_logits": lambda t: nm.adjust_logits(t, bias=torch.ones(64, device="cuda"), out=t),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_saved_tensor_that_was_written_is_noticed(name):
    x = randn(64, 8, seed=4).requires_grad_()
    h = x * 2
    loss = (h * h).float().sum()  # saves h
    before = h._version
    CALLS[name](h.detach())
    assert h._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inputs_and_results_of_their_own_keep_theirs():
    t = randn(64, 8, seed=4)
    y = nm.spmm_act(*pair(), t, layout="blocked", rows=64)
    nm.adjust_logits(t)
    nm.grad_norm([t])
    assert t._version == 0 and y._version == 0


def test_under_inference_mode():
    with torch.inference_mode():
        for call in CALLS.values():
            call(randn(64, 8, seed=5))
