"""Host-only checks of the 4-bit, cross-entropy and orthogonalised-update calls: sizes, and
refusal of bad arguments before a device is touched.  No kernel is launched here."""
import ctypes
import os

import pytest
import torch

import masking_sparse_gemm_amd as nm

pytestmark = pytest.mark.skipif(not os.path.exists(nm.LIB_PATH), reason="libnm.so not built")

P = ctypes.c_void_p(1 << 20)          # aligned, never read
ODD = ctypes.c_void_p((1 << 20) + 8)  # not aligned
BIG = 1 << 60


def far(i):
    """Distinct aligned addresses 2^40 apart."""
    return ctypes.c_void_p((i + 1) << 40)


def st(code):
    return nm.STATUS[code]


def test_sizes():
    L = nm.lib()
    assert L.nm_codes_bytes(1, 1) == 1024 and L.nm_codes_bytes(17, 129) == 4096
    assert L.nm_codes_bytes(0, 5) == 0 and L.nm_codes_bytes(-1, 5) == 0
    assert L.nm_scales_bytes(17, 129, 64) == 2 * 3 * 32
    assert L.nm_scales_bytes(17, 129, 48) == 0
    assert L.nm_matvec_workspace_bytes(4096, 4096, 1, 0) == 0
    assert L.nm_matvec_workspace_bytes(-1, 4096, 2, 0) == 0
    assert L.nm_matvec_workspace_bytes(128, 65536, 2, 1) > 0    # X beyond the LDS: slices to be joined
    assert L.nm_matvec_workspace_bytes(128, 4096, 16, 0) == 0
    assert L.nm_xent_workspace_bytes(0, 8, 1) == 0
    assert L.nm_xent_grad_workspace_bytes(1 << 31, 8, 1) == 0
    assert L.nm_orthogonalize_workspace_bytes(8, 8, nm.NM_I8) == 0
    assert L.nm_orthogonalize_workspace_bytes(8, 8, nm.NM_BF16) > 0
    # a piece of the vocabulary bounds the gradient's workspace: it does not grow with V
    a = L.nm_xent_grad_workspace_bytes(1 << 17, 1024, 4096)
    assert a == L.nm_xent_grad_workspace_bytes(1 << 18, 1024, 4096) < 2 * (1 << 17) * 4096


def quantize(W=P, dt=nm.NM_BF16, R=16, C=128, layout=0, group=64, codes=far(1), scales=far(2),
             sdt=nm.NM_BF16):
    return st(nm.lib().nm_quantize(W, dt, R, C, layout, group, codes, scales, sdt, None))


def test_quantize_refusals():
    assert quantize(dt=nm.NM_I8) == "dtype" and quantize(sdt=nm.NM_F32) == "dtype"
    assert quantize(R=-1) == "shape" and quantize(R=1 << 30, C=1 << 30) == "shape"
    assert quantize(group=48) == "unsupported" and quantize(group=0) == "unsupported"
    assert quantize(layout=1, C=48) == "layout" and quantize(layout=2) == "layout"
    assert quantize(W=None) == quantize(codes=None) == quantize(scales=None) == "null"
    assert quantize(W=ODD) == quantize(codes=ODD) == quantize(scales=ODD) == "align"
    assert quantize(codes=P) == quantize(scales=far(1)) == "alias"
    assert quantize(R=0, W=None, codes=None, scales=None) == "ok"


def dequantize(codes=far(1), scales=far(2), sdt=nm.NM_F16, R=16, C=128, layout=0, group=64, W=P):
    return st(nm.lib().nm_dequantize(codes, scales, sdt, R, C, layout, group, W, None))


def test_dequantize_refusals():
    assert dequantize(sdt=nm.NM_F32) == "dtype" and dequantize(C=-1) == "shape"
    assert dequantize(group=256) == "unsupported" and dequantize(layout=1, C=33) == "layout"
    assert dequantize(W=None) == "null" and dequantize(codes=ODD) == "align"
    assert dequantize(W=far(1)) == "alias" and dequantize(C=0) == "ok"


def matvec(codes=far(1), scales=far(2), meta=None, R=16, K=128, group=64, X=far(3), T=2,
           dt=nm.NM_BF16, Y=far(4), ydt=nm.NM_BF16, ws=far(5), n=BIG):
    return st(nm.lib().nm_matvec(codes, scales, meta, R, K, group, X, T, dt, Y, ydt, ws, n, None))


def test_matvec_refusals():
    assert matvec(dt=nm.NM_F32, ydt=nm.NM_F32) == "dtype" and matvec(ydt=nm.NM_F16) == "dtype"
    assert matvec(R=1 << 26, K=1) == matvec(K=1 << 25) == "shape"
    assert matvec(T=-1) == matvec(T=1 << 20) == matvec(K=-1) == "shape"
    assert matvec(group=16) == "unsupported" and matvec(meta=far(6), K=96) == "layout"
    assert matvec(codes=None) == matvec(X=None) == matvec(Y=None) == "null"
    assert matvec(ws=None, K=65536) == "null"
    assert matvec(X=ODD) == matvec(ws=ODD) == matvec(meta=ODD) == "align"
    assert matvec(n=100, K=65536) == "scratch"
    assert matvec(Y=far(3)) == matvec(Y=far(5), K=65536) == matvec(ws=far(1), K=65536) == "alias"
    assert matvec(meta=far(4)) == "alias"
    assert matvec(R=0) == matvec(T=0) == "ok"


def xent(W=far(1), X=far(2), dt=nm.NM_BF16, V=100, K=64, T=8, y=far(3), loss=far(4), lse=far(5),
         ws=far(6), n=BIG):
    return st(nm.lib().nm_xent(W, X, dt, V, K, T, y, loss, lse, ws, n, None))


def test_xent_refusals():
    assert xent(dt=nm.NM_F32) == "dtype"
    assert xent(V=0) == xent(V=1 << 31) == xent(K=1 << 22) == xent(T=1 << 22) == xent(T=-1) == "shape"
    assert xent(V=1 << 20, T=1 << 16) == xent(K=1 << 18, T=1 << 18) == "shape"
    assert xent(W=None) == xent(y=None) == xent(lse=None) == xent(ws=None) == "null"
    assert xent(X=ODD) == xent(y=ODD) == xent(ws=ODD) == "align"
    assert xent(n=64) == "scratch"
    assert xent(loss=far(5)) == xent(lse=far(1)) == xent(ws=far(2)) == "alias"
    assert xent(T=0, X=None, y=None, loss=None, lse=None, ws=None, n=0) == "ok"


def xent_grad(W=far(1), X=far(2), dt=nm.NM_BF16, V=100, K=64, T=8, y=far(3), lse=far(4), g=far(5),
              dW=far(6), dX=far(7), ws=far(8), n=BIG):
    return st(nm.lib().nm_xent_grad(W, X, dt, V, K, T, y, lse, g, dW, dX, ws, n, None))


def test_xent_grad_refusals():
    assert xent_grad(dt=nm.NM_FP8) == "dtype" and xent_grad(V=0) == "shape"
    assert xent_grad(g=None) == xent_grad(dW=None) == xent_grad(dX=None) == "null"
    assert xent_grad(lse=ODD) == xent_grad(g=ODD) == xent_grad(dX=ODD) == "align"
    assert xent_grad(n=1000) == "scratch"
    assert xent_grad(dW=far(1)) == xent_grad(dX=far(2)) == xent_grad(dX=far(6)) == "alias"
    assert xent_grad(dW=far(5)) == xent_grad(ws=far(4)) == "alias"
    assert xent_grad(K=0) == xent_grad(V=0, T=0) == "ok"


def orth(G=far(1), dt=nm.NM_BF16, R=64, K=64, steps=5, eps=0.0, out=far(2), ws=far(3), n=BIG):
    return st(nm.lib().nm_orthogonalize(G, dt, R, K, steps, eps, out, ws, n, None))


def test_orthogonalize_refusals():
    assert orth(dt=nm.NM_I8) == "dtype"
    assert orth(R=-1) == orth(K=1 << 22) == orth(steps=0) == orth(steps=101) == "shape"
    assert orth(eps=-1.0) == orth(eps=float("nan")) == "shape"
    assert orth(G=None) == orth(out=None) == orth(ws=None) == "null"
    assert orth(G=ODD) == orth(out=ODD) == "align" and orth(n=10) == "scratch"
    assert orth(ws=far(1)) == orth(ws=far(2)) == "alias"
    assert orth(out=ctypes.c_void_p(far(1).value + 16)) == "alias"
    assert orth(R=0, G=None, out=None, ws=None, n=0) == "ok"


def test_binding_refuses_what_is_not_on_a_gpu_or_has_no_kernel():
    w = torch.zeros(16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nm.quantize(w)
    with pytest.raises(ValueError):
        nm.quantize(w, group=16)
    with pytest.raises(ValueError):
        nm.xent(w, w.t().contiguous(), torch.zeros(16, dtype=torch.int64))
    with pytest.raises(ValueError):
        nm.orthogonalize(w)
    with pytest.raises(ValueError):
        nm.matvec(torch.zeros(1, 1, 64, 4, dtype=torch.int32), torch.zeros(1, 1, 16), w, rows=16)
    assert nm.code_shapes(17, 129, 32) == ((2, 2, 64, 4), (2, 5, 16))
