"""The smooth activations' negative tails in fp32, relative to the value: what is left of 1 there is an
exponential, whose argument's rounding is the error that grows."""
import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests import act_ref as ref

pytestmark = pytest.mark.gpu

# to where e^-a is a normal number of fp32
ENDS = {"silu": 85.0, "gelu": 12.8, "gelu_tanh": 9.0}


def tail(z, act):
    """(act(z), the exponent a of e^-a in it), 64 bits."""
    if act == "silu":
        return z * torch.sigmoid(z), z.abs()
    if act == "gelu":
        # (1 + erf, which torch.special.ndtr computes, is 0 below -8.3 in 64 bits as well)
        return z * torch.erfc(-z * 0.5 ** 0.5) / 2, z * z / 2
    a = (2 * ref.ROOT * (z + 0.044715 * z ** 3)).abs()
    return z / (1 + torch.exp(a)), a


@pytest.mark.parametrize("act", ENDS)
@pytest.mark.parametrize("K", [0, 64])
def test_negative_tail_keeps_its_relative_accuracy(act, K):
    """Four roundings at most of the argument, each 2^-24 of it; the polynomial (4e-7), the exponential and
    the reciprocal (2^-23 each) and three products (2^-24 each) are 2^-20 together."""
    z = -torch.linspace(0.01, ENDS[act], 4000)
    w = torch.zeros(4000, K, device="cuda")
    values, meta = nm.compress(w, 2, 4)
    X = torch.zeros(K, 3, device="cuda")
    y = nm.spmm_act(values, meta, X, bias=z.cuda(), act=act).cpu().double()
    want, a = tail(z.double(), act)
    bound = (2.0 ** -20 + 2.0 ** -22 * a) * want.abs()
    assert bool(((y - want[:, None]).abs() <= bound[:, None]).all()), \
        float(((y[:, 0] - want).abs() / bound).max())
