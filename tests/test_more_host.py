"""Host-only checks of the epilogue, clipping and logits calls: sizes, and refusal of bad arguments
before a device is touched.  No kernel is launched here."""
import ctypes
import os

import pytest
import torch

import masking_sparse_gemm_amd as nm
from tests.test_lm_host import BIG, ODD, far, st

pytestmark = pytest.mark.skipif(not os.path.exists(nm.LIB_PATH), reason="libnm.so not built")

BF, F16, F32, I8, FP8 = nm.NM_BF16, nm.NM_F16, nm.NM_F32, nm.NM_I8, nm.NM_FP8


def test_sizes():
    L = nm.lib()
    act = L.nm_spmm_act_workspace_bytes
    assert act(32, 72, 3, 8, 8, BF) == 0                 # rows of X are whole pieces
    assert act(32, 72, 3, 8, 7, BF) == 72 * 8 * 2 // 256 * 256 + 256
    assert act(32, 72, 3, 8, 7, F32) == 72 * 8 * 4 and act(32, 72, 3, 8, 17, I8) == 72 * 32
    assert act(32, 60, 2, 4, 7, BF) == 64 * 16 * 2       # few tokens: X turned, in whole steps
    assert act(32, 60, 2, 4, 7, F32) == 64 * 16 * 4 and act(32, 60, 1, 2, 7, I8) == 64 * 16 * 2
    assert act(32, 64, 2, 4, 7, BF) == act(32, 64, 1, 2, 7, I8) == act(32, 64, 2, 4, 1, F32) == 0  # as it lies
    assert act(1000, 1024, 2, 4, 517, BF) == 1024 * 544 * 2   # many workgroups read it: turned
    assert act(8192, 4096, 2, 4, 2048, BF) == 0          # many: as it lies
    assert act(32, -4, 2, 4, 7, BF) == act(32, 64, 2, 4, 7, 9) == act(32, 64, 5, 4, 7, BF) == 0
    need = L.nm_spmm_act_grad_workspace_bytes
    assert need(64, 64, 64, 0, 1, 0, 0) == 0                       # dW = dY X^T as they lie
    assert need(64, 64, 64, 0, 1, 1, 0) == 64 * 64 * 2             # the dense W
    assert need(64, 64, 64, 3, 1, 0, 0) == 64 * 64 * 2             # dZ
    assert need(64, 64, 64, 3, 1, 0, 1) == 0                       # dZ is a result
    assert need(64, 64, 64, 3, 0, 0, 1) == 0 == need(64, 64, 64, 3, 0, 0, 0)
    assert need(65, 64, 64, 0, 1, 0, 0) == 128 * 64 * 2            # padded rows
    assert need(64, 64, 64, 6, 1, 1, 0) == need(1 << 22, 64, 64, 0, 1, 1, 0) == 0
    counts = (ctypes.c_int64 * 3)(0, 5, 1 << 30)
    at = ctypes.addressof(counts)
    assert L.nm_grad_norm_workspace_bytes(at, 3) == 2048 * 8
    assert L.nm_grad_norm_workspace_bytes(at, 1) == L.nm_grad_norm_workspace_bytes(None, 0) == 0
    assert L.nm_adjust_logits_workspace_bytes(32000, 1, 2000) == 0
    assert L.nm_adjust_logits_workspace_bytes(32000, 64, 64 * 100000) == 32000 * 64 * 4
    assert L.nm_adjust_logits_workspace_bytes(32000, 1 << 20, 8) == 0


def spmm_act(values=far(1), meta=far(2), R=32, K=128, n=2, m=4, layout=1, X=far(3), T=16, dt=BF,
             scale=None, bias=far(4), act=3, residual=far(5), Z=far(6), Y=far(7), ydt=BF, ws=far(8),
             size=BIG):
    return st(nm.lib().nm_spmm_act(values, meta, R, K, n, m, layout, X, T, dt, scale, bias, act,
                                   residual, Z, Y, ydt, ws, size, None))


def test_spmm_act_refusals():
    assert spmm_act(dt=9) == spmm_act(ydt=F16) == spmm_act(ydt=I8) == "dtype"
    assert spmm_act(scale=far(9)) == "dtype"                       # of 16 bits
    assert spmm_act(dt=I8, Z=None, ydt=nm.NM_I32) == spmm_act(dt=FP8) == "dtype"
    assert spmm_act(n=5) == spmm_act(m=3) == "pattern"
    assert spmm_act(K=130) == spmm_act(T=-1) == spmm_act(R=-1) == spmm_act(T=1 << 40) == "shape"
    assert spmm_act(dt=I8, Z=None, K=1 << 17) == "shape"
    assert spmm_act(K=96) == spmm_act(layout=5) == "layout"
    assert spmm_act(act=6) == spmm_act(act=-1) == "unsupported"
    assert spmm_act(dt=I8, Z=None, n=1, m=8, ydt=F32) == "unsupported"
    assert spmm_act(values=None) == spmm_act(meta=None) == spmm_act(X=None) == spmm_act(Y=None) == "null"
    many = dict(R=1000, K=1024, T=517)                             # (whose X is turned)
    assert spmm_act(ws=None, **many) == "null" and spmm_act(size=100, **many) == "scratch"
    for name in ("values", "meta", "X", "bias", "residual", "Z", "Y"):
        assert spmm_act(**{name: ODD}) == "align", name
    assert spmm_act(ws=ODD) == "align"
    assert spmm_act(dt=I8, Z=None, scale=ODD, ydt=F32) == "align"
    for name in ("values", "meta", "X", "bias", "Z"):
        assert spmm_act(**{name: far(7)}) == "alias", name
    assert spmm_act(Z=far(5)) == spmm_act(ws=far(3), **many) == spmm_act(ws=far(6), **many) == "alias"
    assert spmm_act(residual=ctypes.c_void_p(far(7).value + 64)) == "alias"
    assert spmm_act(residual=far(7)) == "device"                   # in place: as far as a GPU
    assert spmm_act(bias=None, residual=None, Z=None) == "device"
    assert spmm_act(R=0) == spmm_act(T=0) == "ok"


def grad(values=far(1), meta=far(2), R=32, K=128, n=2, m=4, layout=1, X=far(3), T=16, dt=BF, act=3,
         Z=far(4), dY=far(5), dW=far(6), dX=far(7), db=far(8), dZ=far(9), ws=far(10), size=BIG):
    return st(nm.lib().nm_spmm_act_grad(values, meta, R, K, n, m, layout, X, T, dt, act, Z, dY, dW,
                                        dX, db, dZ, ws, size, None))


def test_spmm_act_grad_refusals():
    assert grad(dt=F32) == grad(dt=I8) == "dtype" and grad(m=5) == "pattern"
    assert grad(R=1 << 22) == grad(T=1 << 22) == grad(K=1 << 22) == grad(T=-1) == grad(K=6) == "shape"
    assert grad(R=1 << 20, T=1 << 20) == "shape"
    assert grad(K=100) == "layout" and grad(act=7) == "unsupported"
    assert grad(Z=None) == grad(dY=None) == grad(X=None) == grad(values=None) == grad(meta=None) == "null"
    assert grad(ws=None) == "null" and grad(size=64) == "scratch"
    for name in ("values", "meta", "X", "Z", "dY", "dW", "dX", "db", "dZ", "ws"):
        assert grad(**{name: ODD}) == "align", name
    for name in ("dW", "dX", "db", "dZ", "ws"):
        for other in (1, 2, 3, 4, 5):
            assert grad(**{name: far(other)}) == "alias", (name, other)
    assert grad(dW=far(7)) == grad(dZ=far(8)) == "alias"
    # what is not wanted does not need its inputs
    assert grad(values=None, meta=None, dX=None) == "device"
    assert grad(values=None, meta=None, X=None, dX=None, dW=None, ws=None, size=0) == "device"
    assert grad(act=0, Z=None) == "device"
    assert grad(R=0, K=0, T=0) == "ok"


def matvec_act(codes=far(1), scales=far(2), meta=None, R=16, K=128, group=64, X=far(3), T=2, dt=BF,
               bias=far(4), act=1, residual=far(5), Y=far(6), ydt=BF, ws=far(7), size=BIG):
    return st(nm.lib().nm_matvec_act(codes, scales, meta, R, K, group, X, T, dt, bias, act, residual,
                                     Y, ydt, ws, size, None))


def test_matvec_act_refusals():
    assert matvec_act(dt=F32, ydt=F32) == matvec_act(ydt=F16) == "dtype"
    assert matvec_act(T=1 << 20) == matvec_act(R=1 << 26) == "shape"
    assert matvec_act(group=48) == matvec_act(act=6) == "unsupported"
    assert matvec_act(meta=far(9), K=96) == "layout"
    assert matvec_act(codes=None) == matvec_act(X=None) == matvec_act(Y=None) == "null"
    for name in ("codes", "scales", "X", "bias", "residual", "Y"):
        assert matvec_act(**{name: ODD}) == "align", name
    assert matvec_act(K=65536, size=10) == "scratch" and matvec_act(K=65536, ws=None) == "null"
    for name in ("codes", "scales", "X", "bias"):
        assert matvec_act(**{name: far(6)}) == "alias", name
    assert matvec_act(residual=ctypes.c_void_p(far(6).value + 16)) == "alias"
    assert matvec_act(residual=far(6)) == matvec_act(bias=None, residual=None) == "device"
    assert matvec_act(R=0) == matvec_act(T=0) == "ok"


def clip(pairs, counts, dts, most=1.0, given=None, norm=far(100), ws=far(101), size=BIG, only_norm=False):
    n = len(counts)
    grads = (ctypes.c_void_p * n)(*[a for a, _ in pairs])
    outs = (ctypes.c_void_p * n)(*[b for _, b in pairs])
    held = grads, outs, (ctypes.c_int64 * n)(*counts), (ctypes.c_int * n)(*dts)
    g, o, c, d = (ctypes.addressof(x) for x in held)
    L = nm.lib()
    if only_norm:
        return st(L.nm_grad_norm(g, c, d, n, norm, ws, size, None))
    return st(L.nm_clip_grads(g, o, c, d, n, most, given, norm, ws, size, None))


def test_clip_refusals():
    a, b = far(1).value, far(2).value
    one = [(a, a)]
    for only in (False, True):
        assert clip(one, [8], [I8], only_norm=only) == "dtype"
        assert clip(one, [-1], [F32], only_norm=only) == clip(one, [1 << 40], [F32], only_norm=only) == "shape"
        assert clip([(None, None)], [8], [F32], only_norm=only) == "null"
        assert clip([(a + 2, a + 2)], [8], [F32], only_norm=only) == "align"
        assert clip([(a + 1, a + 1)], [8], [BF], only_norm=only) == "align"
        assert clip([(a + 2, a + 2)], [8], [BF], only_norm=only) == "device"
        assert clip(one, [8], [BF], norm=None, only_norm=only) == "null"
        assert clip(one, [8], [BF], norm=ctypes.c_void_p(6), only_norm=only) == "align"
        assert clip(one, [8], [BF], size=16, only_norm=only) == "scratch"
        assert clip(one, [8], [BF], ws=None, only_norm=only) == "null"
        assert clip(one, [8], [BF], norm=ctypes.c_void_p(a + 4), only_norm=only) == "alias"
        assert clip(one, [8], [BF], ws=far(1), only_norm=only) == "alias"
    assert clip(one, [8], [BF], most=-1.0) == clip(one, [8], [BF], most=float("nan")) == "shape"
    assert clip([(a, None)], [8], [BF]) == "null"
    # read twice is fine, written twice is not
    assert clip([(a, a), (a, a)], [8, 8], [BF, BF], only_norm=True) == "device"
    assert clip([(a, a), (a, a)], [8, 8], [BF, BF]) == "alias"
    assert clip([(a, b), (a, b + 16)], [8, 8], [BF, BF]) == "device"
    assert clip([(a, b), (a, b + 14)], [8, 8], [BF, BF]) == "alias"
    assert clip([(a, b), (b + 8, b + 64)], [8, 8], [BF, BF]) == "alias"   # an output over an input
    assert clip([(a, a + 2)], [8], [BF]) == "alias"                       # shifted by one
    assert clip([(a, a), (b, b), (a + 16, a + 16)], [8, 0, 8], [BF, F32, BF]) == "device"
    # a long range that spans later ones
    assert clip([(a, a), (a + 400, a + 400), (a + 200, b)], [100, 8, 8], [F32] * 3) == "alias"
    # a given norm needs no workspace
    assert clip(one, [8], [BF], given=far(50), norm=None, ws=None, size=0) == "device"
    assert clip(one, [8], [BF], given=ctypes.c_void_p(a + 4), norm=None) == "alias"


def logits(x=far(1), dt=F32, V=100, T=3, tokens=far(2), count=10, starts=far(3), prompts=far(4),
           rep=far(5), pres=far(6), freq=far(7), bias=far(8), each=0, allowed=far(9), out=far(10),
           ws=far(11), size=BIG):
    return st(nm.lib().nm_adjust_logits(x, dt, V, T, tokens, count, starts, prompts, rep, pres, freq,
                                        bias, each, allowed, out, ws, size, None))


def test_adjust_logits_refusals():
    assert logits(dt=I8) == "dtype"
    assert logits(V=-1) == logits(V=1 << 31) == logits(T=1 << 20) == logits(count=-1) == "shape"
    assert logits(V=1 << 30, T=1 << 10) == logits(count=1 << 31) == "shape"
    assert logits(x=None) == logits(out=None) == logits(starts=None) == "null"
    for name in ("x", "tokens", "starts", "prompts", "rep", "pres", "freq", "bias", "allowed", "out"):
        assert logits(**{name: ODD}) == "align", name
    for name in ("tokens", "starts", "prompts", "rep", "pres", "freq", "bias", "allowed"):
        assert logits(**{name: far(10)}) == "alias", name
    assert logits(V=32000, T=64, count=64 * 100000, size=100) == "scratch"
    assert logits(V=32000, T=64, count=64 * 100000, ws=None) == "null"
    assert logits(V=32000, T=64, count=64 * 100000, ws=far(1)) == "alias"
    assert logits(out=ctypes.c_void_p(far(1).value + 16)) == "alias"
    assert logits(out=far(1)) == "device"
    assert logits(tokens=None, starts=None, prompts=None, rep=None, pres=None, freq=None, bias=None,
                  allowed=None, ws=None, size=0) == "device"
    assert logits(V=0) == logits(T=0) == "ok"


def test_binding_refuses_what_is_not_on_a_gpu():
    w = torch.zeros(16, 64, dtype=torch.bfloat16)
    v, m = torch.zeros(16, 32, dtype=torch.bfloat16), torch.zeros(16, 4, dtype=torch.int32)
    for call in (lambda: nm.spmm_act(v, m, w), lambda: nm.spmm_act_grad(v, m, w, w),
                 lambda: nm.grad_norm([w]), lambda: nm.clip_grads(w, 1.0),
                 lambda: nm.adjust_logits(w.float()),
                 lambda: nm.matvec_act(torch.zeros(1, 1, 64, 4, dtype=torch.int32),
                                       torch.zeros(1, 1, 16), w, rows=16)):
        with pytest.raises(ValueError):
            call()
