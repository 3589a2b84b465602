"""Host-only checks at the limits of the epilogue, gradient, clipping and logits calls."""
import os
import subprocess

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


def test_a_launch_of_the_thin_kernel_has_fewer_than_2_32_work_items(tmp_path):
    """Whatever the shape that the plan takes: one direct column launches 16 rows a workgroup."""
    (tmp_path / "rule.cpp").write_text(r"""
#include <cstdio>
#include "nm_tiles.h"
int main() {
  const int patterns[][2] = {{2, 4}, {1, 2}, {1, 4}, {4, 8}};
  long thin = 0, most = 0;
  for (const auto& p : patterns)
    for (int elem : {1, 2, 4})
      for (long K : {8L, 64L, 128L, 256L, 1024L})
        for (long T : {1L, 2L, 16L, 17L, 33L, 512L, 4096L})
          for (int bit = 20; bit <= 36; ++bit)
            for (long d : {-17L, -16L, -1L, 0L, 1L, 16L}) {
              const long R = (1L << bit) + d;
              if (!nm::thin_preferred(R, K, p[0], p[1], T, elem)) continue;
              ++thin;
              const nm::ThinPlan plan(R, K, T, p[1], elem == 4);
              const long rows = T == 1 && plan.direct ? 16 : 16 * plan.rg;
              const long items = (R + rows - 1) / rows * 512;
              if (items > most) most = items;
            }
  std::printf("%ld %d\n", thin, most < (1L << 32));
}
""")
    csrc = os.path.join(os.path.dirname(nm.LIB_PATH), "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(tmp_path / "rule.cpp"), "-o", str(tmp_path / "rule")],
                   check=True)
    thin, fits = subprocess.run([str(tmp_path / "rule")], check=True, capture_output=True,
                                text=True).stdout.split()
    assert int(thin) > 100 and fits == "1"


def test_a_launch_of_the_logits_kernel_has_fewer_than_2_32_work_items(tmp_path):
    """Over all that the call accepts: V < 2^31, T < 2^20, V T < 2^36, with and without tokens."""
    (tmp_path / "rule.cpp").write_text(r"""
#include <cstdio>
#include "nm_tiles.h"
int main() {
  long seen = 0, wrong = 0;
  for (int bit = 0; bit <= 31; ++bit)
    for (long dv : {-1L, 0L, 1L})
      for (int t = 0; t <= 20; ++t)
        for (long d : {-1L, 0L, 1L})
          for (long count : {0L, 1L, 1000L, 1L << 20, (1L << 31) - 1}) {
            const long V = (1L << bit) + dv, T = (1L << t) + d;
            if (V < 1 || T < 1 || V >= 1L << 31 || T >= 1L << 20 || V * T >= 1L << 36) continue;
            const nm::LogitsPlan p(V, T, count);
            ++seen;
            const long words = (1L << p.log_cells) >> p.log_cols, cols = 1L << p.log_cols;
            const bool fits = p.threads <= nm::kLogitsThreads && p.grid_v * p.threads < 1L << 32 &&
                              p.blocks_t < 65536 && p.grid_z < 65536 && p.grid_z >= 1;
            const bool covers = p.grid_v * p.grid_z * words >= V && p.blocks_t * cols >= T &&
                                p.grid_v * (p.grid_z - 1) * words < V;
            const bool holds = (1 << p.log_cells) <= nm::kLogitsEach * p.threads && words % 32 == 0 &&
                               cols <= 32 && p.copies * cols * (words + 1) <= 8448;
            if (!fits || !covers || !holds) ++wrong;
          }
  std::printf("%ld %ld\n", seen, wrong);
}
""")
    csrc = os.path.join(os.path.dirname(nm.LIB_PATH), "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(tmp_path / "rule.cpp"), "-o", str(tmp_path / "rule")],
                   check=True)
    seen, wrong = subprocess.run([str(tmp_path / "rule")], check=True, capture_output=True,
                                 text=True).stdout.split()
    assert int(seen) > 5000 and wrong == "0"


def test_a_copy_of_X_for_the_thin_kernel_has_fewer_than_2_32_work_items(tmp_path):
    (tmp_path / "rule.cpp").write_text(r"""
#include <cstdio>
#include "nm_tiles.h"
int main() {
  long copies = 0, most = 0;
  for (int bit = 20; bit < 36; ++bit)
    for (long d : {-60L, 4L, 8L, 64L})
      for (long T : {1L, 2L, 33L, 4096L})
        for (long R : {1L, 3L, 16L})
          for (int elem : {1, 2, 4}) {
            const long K = (1L << bit) + d;
            const nm::ThinPlan plan(R, K, T, 4, elem == 4);
            if (plan.direct || !nm::thin_preferred(R, K, 2, 4, T, elem)) continue;
            ++copies;
            if ((K + 63) / 64 * 256 > most) most = (K + 63) / 64 * 256;
          }
  std::printf("%ld %d\n", copies, most < (1L << 32));
}
""")
    csrc = os.path.join(os.path.dirname(nm.LIB_PATH), "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(tmp_path / "rule.cpp"), "-o", str(tmp_path / "rule")],
                   check=True)
    copies, fits = subprocess.run([str(tmp_path / "rule")], check=True, capture_output=True,
                                  text=True).stdout.split()
    assert int(copies) > 50 and fits == "1"


def test_long_rows_of_bytes_take_the_thin_kernel(tmp_path):
    """The sizes of test_gpu_act_exact.py: more than sixteen steps of 64 to each of eight waves."""
    (tmp_path / "rule.cpp").write_text(r"""
#include <cstdio>
#include "nm_tiles.h"
int main() {
  const int patterns[][2] = {{2, 4}, {1, 2}, {1, 4}, {4, 8}};
  const long sizes[][3] = {{33, (1 << 17) - 64, 1}, {33, (1 << 17) - 64, 20}, {20, (1 << 17) - 24, 20},
                           {20, (1 << 17) - 24, 1}};
  int thin = 0;
  for (const auto& p : patterns)
    for (const auto& s : sizes) thin += nm::thin_preferred(s[0], s[1], p[0], p[1], s[2], 1);
  std::printf("%d\n", thin);
}
""")
    csrc = os.path.join(os.path.dirname(nm.LIB_PATH), "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(tmp_path / "rule.cpp"), "-o", str(tmp_path / "rule")],
                   check=True)
    assert subprocess.run([str(tmp_path / "rule")], check=True, capture_output=True, text=True).stdout == "16\n"


def test_a_gradient_in_fp16_is_refused_the_other_types_workspace():
    from tests.test_more_host import grad

    sizes = dict(R=32, K=128, T=16, act=3)
    L = nm.lib()
    plain = L.nm_spmm_act_grad_workspace_bytes(32, 128, 16, 3, 1, 1, 1)
    typed = L.nm_spmm_act_grad_dt_workspace_bytes(32, 128, 16, nm.NM_F16, 3, 1, 1, 1)
    assert grad(dt=nm.NM_F16, size=plain, **sizes) == grad(dt=nm.NM_F16, size=typed - 1, **sizes) == "scratch"
    assert grad(dt=nm.NM_F16, size=typed, **sizes) == grad(dt=nm.NM_BF16, size=plain, **sizes) == "device"
    assert grad(dt=nm.NM_F16, size=plain, **dict(sizes, act=1)) == "device"
