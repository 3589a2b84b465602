"""64-bit references of a product's epilogue and its gradient, with bounds on what fp32 sums and single
roundings may add, for the tests of spmm_act, spmm_act_grad and matvec_act (no kernel of the library
is used here)."""
from __future__ import annotations

import math

import torch

ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")
ROOT = math.sqrt(2 / math.pi)
# half a step of a type, relative to the value, and half of its smallest step
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.float16, torch.bfloat16)}
LEAST = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
F32 = 2.0 ** -24


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "relu2":
        return z.clamp(min=0) ** 2
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(ROOT * (z + 0.044715 * z ** 3)))
    return z


def slope(z, name):
    if name in ("relu", "relu2"):
        return (z > 0).double() * (2 * z if name == "relu2" else 1)
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * torch.sigmoid(-z)
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(ROOT * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * ROOT * (1 + 0.134145 * z * z)
    return torch.ones_like(z)


def rounding(y, dtype):
    """Half a step at y."""
    return HALF[dtype] * y.abs() + LEAST[dtype]


def sum_bound(terms, absolute):
    """What a sum of `terms` fp32 products in any order may be off, `absolute` the sum of their sizes:
    each of the products, additions and the epilogue's few steps rounds once."""
    return (terms + 4) * F32 * absolute


def after_act(z, off, name):
    """How far act may be off where its argument is off by `off`: no slope is above 1.13 but relu2's,
    and its own few steps (exponential, reciprocal, polynomial) are off by at most 2^-20 of z."""
    if name == "none":
        return off
    if name == "relu2":
        return (2 * z.abs() + off) * off + 2 * F32 * z * z
    return 1.13 * off + 2.0 ** -20 * z.abs()


def epilogue(sums, off, bias, name, residual, y_dtype, z_dtype=None):
    """(Y, its bound, Z, its bound) of 64-bit sums that fp32 knows to `off`."""
    z = sums if bias is None else sums + bias.double()[:, None]
    off = off + 2 * F32 * z.abs()
    y = act(z, name)
    y_off = after_act(z, off, name)
    if residual is not None:
        y = y + residual.double()
    y_off = y_off + F32 * y.abs() + rounding(y, y_dtype)
    # a result off by `off` before rounding rounds to at most half a step more of what it became
    y_off = y_off * (1 + 2 * HALF[y_dtype])
    if z_dtype is None:
        return y, y_off, None, None
    return y, y_off, z, (off + rounding(z, z_dtype)) * (1 + 2 * HALF[z_dtype])


SLOPE_OFF = 2.0 ** -18   # of a slope: (1 - s) is known to 2^-24 and meets factors of at most 30


def gradient(W, X, Z, dY, name, dtype):
    """{name: (value, bound)} of dZ, dbias, dW and dX in 64 bits; W dense (or None), X and dY the
    inputs as they are stored."""
    dy = dY.double()
    z = torch.zeros_like(dy) if Z is None else Z.double()
    dz = dy * slope(z, name)
    exact = name in ("none", "relu")
    size = dy.abs() * (1 + (z.abs() if name == "relu2" else 0))
    off = torch.zeros_like(dz) if exact else SLOPE_OFF * size
    T, R = dz.shape[1], dz.shape[0]
    out = dict(dZ=(dz, (off + (0 if exact else rounding(dz, dtype))) * (1 + 2 * HALF[dtype])))
    out["dbias"] = (dz.sum(1), off.sum(1) + sum_bound(T, dz.abs().sum(1)))
    dz_off = out["dZ"][1]
    if X is not None:
        x = X.double()
        v = dz @ x.t()
        b = dz_off @ x.abs().t() + sum_bound(T, dz.abs() @ x.abs().t())
        out["dW"] = (v, (b + rounding(v, dtype)) * (1 + 2 * HALF[dtype]))
    if W is not None:
        w = W.double()
        v = w.t() @ dz
        b = w.abs().t() @ dz_off + sum_bound(R, w.abs().t() @ dz.abs())
        out["dX"] = (v, (b + rounding(v, dtype)) * (1 + 2 * HALF[dtype]))
    return out


def check(got, want, bound, what):
    """Every finite entry within its bound; the others equal."""
    g = got.double().cpu()
    w, b = want.cpu(), bound.cpu()
    assert g.shape == w.shape, (what, g.shape, w.shape)
    fine = torch.isfinite(w)
    assert torch.equal(torch.isnan(g), torch.isnan(w)), what
    same = g[~fine & ~torch.isnan(w)] == w[~fine & ~torch.isnan(w)]
    assert bool(same.all()), what
    over = ((g - w).abs() - b)[fine]
    if over.numel():
        assert float(over.max()) <= 0, (what, "off by", float((g - w)[fine].abs().max()), "over",
                                       float(over.max()))
