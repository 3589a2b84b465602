"""Host-only checks of the largest sizes that nm_matvec takes.  No kernel is launched here: the
refused calls stop at the checks of their sizes."""
import ctypes
import os

import pytest

import masking_sparse_gemm_amd as nm

pytestmark = pytest.mark.skipif(not os.path.exists(nm.LIB_PATH), reason="libnm.so not built")


def far(i):
    """Distinct aligned addresses 2^40 apart, never read."""
    return ctypes.c_void_p((i + 1) << 40)


def matvec(R, K, T, meta=None):
    return nm.STATUS[nm.lib().nm_matvec(far(1), far(2), meta, R, K, 64, far(3), T, nm.NM_BF16, far(4),
                                        nm.NM_BF16, far(5), 1 << 60, None)]


@pytest.mark.parametrize("R,K,T", [(1 << 24, 4095, 1 << 10), (1 << 20, 1 << 15, 1 << 14),
                                   ((1 << 20) - 15, 1 << 15, (1 << 14) - 31), (1 << 14, 4096, 1 << 20)])
def test_matvec_refuses_results_past_a_launch_of_the_join(R, K, T):
    """The sums of slices are joined by one work-item for each four results: R T of 2^34 (whole 16
    rows and 32 columns) would be 2^32 of them."""
    L = nm.lib()
    if T == 1 << 20:
        T -= 1   # its own limit
    assert matvec(R, K, T) == "shape"
    assert matvec(R, K // 64 * 64, T, far(6)) == "shape"
    assert L.nm_matvec_workspace_bytes(R, K, T, 0) == 0
    assert L.nm_matvec_workspace_bytes(R // 2, K, T, 0) > 0
