"""Host-only checks at the limits of the epilogue, gradient, clipping and logits calls."""
import os

import pytest

import masking_sparse_gemm_amd as nm

pytestmark = pytest.mark.skipif(not os.path.exists(nm.LIB_PATH), reason="libnm.so not built")


def test_workspace_of_a_gradient_by_type():
    L = nm.lib()
    typed = L.nm_spmm_act_grad_dt_workspace_bytes
    plain = L.nm_spmm_act_grad_workspace_bytes
    bf, half = nm.NM_BF16, nm.NM_F16
    for R, K, T in ((64, 64, 64), (65, 64, 63), (1000, 768, 333), (4096, 64, 9)):
        for want in ((1, 0, 0), (0, 1, 0), (1, 1, 1), (0, 0, 1)):
            for act in nm.ACTS.values():
                need = plain(R, K, T, act, *want)
                assert typed(R, K, T, bf, act, *want) == need
                exact = nm.ACTS["relu"] >= act or not (want[0] or want[1])
                assert (typed(R, K, T, half, act, *want) == need) == exact
                assert typed(R, K, T, half, act, *want) >= need
    # dW's copy of dZ, dX's, what brings rows and columns back, the dense W
    assert typed(64, 64, 64, half, 3, 1, 1, 0) == 2 * 64 * 64 * 2 + 2 * 256 + 64 * 64 * 2
    assert typed(64, 64, 64, nm.NM_F32, 3, 1, 1, 0) == typed(64, 64, 64, half, 6, 1, 1, 0) == 0
