"""Which kernel a product with an epilogue takes, by the rule that the library compiles in, and its sizes:
a small C++ program with the header's rule says so on the CPU."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "masking_sparse_gemm_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "nm_tiles.h"
int main(int, char** a) {
  const long R = atol(a[1]), K = atol(a[2]), T = atol(a[5]);
  const int n = atoi(a[3]), m = atoi(a[4]), elem = atoi(a[6]);
  const nm::ThinPlan p(R, K, T, m, elem == 4);
  const nm::SpmmGradCut c(R, K, T, true, true);
  std::printf("%d %d %d %ld %d %d %d %d\n", (int)nm::thin_preferred(R, K, n, m, T, elem), p.rg, p.nt,
              (long)p.Tp, c.tile, c.splits_x, c.splits_w, (int)p.direct);
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    at = tmp_path_factory.mktemp("rule")
    (at / "rule.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(at / "rule.cpp"), "-o", str(at / "rule")],
                   check=True)

    def ask(R, K, n, m, T, elem):
        out = subprocess.run([str(at / "rule"), *map(str, (R, K, n, m, T, elem))], check=True,
                             capture_output=True, text=True).stdout.split()
        return dict(zip(("thin", "rg", "nt", "Tp", "tile", "splits_x", "splits_w", "direct"), map(int, out)))
    return ask


def test_thin_or_tiled(rule):
    assert rule(4096, 4096, 2, 4, 1, 2)["thin"] and rule(1000, 1024, 2, 4, 517, 2)["thin"]
    assert not rule(11008, 4096, 2, 4, 2048, 2)["thin"] and not rule(4096, 11008, 2, 4, 2048, 2)["thin"]
    assert rule(64, 100, 2, 4, 1, 2)["thin"]           # K need not be whole steps
    assert rule(64, 64, 4, 8, 1, 2)["thin"] and not rule(64, 64, 2, 2, 1, 2)["thin"]
    assert rule(4096, 4096, 1, 4, 256, 2)["thin"] and rule(4096, 4096, 2, 4, 512, 4)["thin"]
    assert not rule(16, 64, 2, 4, 1 << 20, 2)["thin"]


def test_sizes_of_the_tiled_kernels_tests(rule):
    for R, K, T in ((2000, 128, 2056), (2000, 128, 2061), (2000, 192, 2061)):
        for n, m in ((2, 4), (1, 2), (1, 4), (4, 8)):
            for elem in (1, 2, 4):
                assert not rule(R, K, n, m, T, elem)["thin"], (R, K, T, n, m, elem)


def test_sizes_of_the_thin_kernels_tests(rule):
    """Every shape of a workgroup, with X turned and as it lies."""
    shape = lambda *a: [rule(*a)[k] for k in ("thin", "rg", "nt", "direct")]
    for n, m in ((2, 4), (1, 2), (1, 4), (4, 8)):
        for elem in (1, 2):
            assert shape(1000, 1024, n, m, 517, elem) == [1, 2, 2, 0]
            assert shape(2048, 1024, n, m, 517, elem) == [1, 2, 4, 0]
            assert shape(77, 192, n, m, 33, elem) == [1, 1, 1, 1]
            assert shape(256, 192, n, m, 1000, elem) == [1, 2, 2, 1]
        assert shape(1000, 1024, n, m, 517, 4) == [1, 1, 1, 0] and shape(77, 192, n, m, 33, 4) == [1, 1, 1, 1]
        assert shape(256, 192, n, m, 2000, 4) == [1, 2, 2, 1]
        assert shape(256, 180, n, m, 2000, 4) == [1, 2, 2, 0]
    assert shape(300, 100, 2, 4, 7, 2) == [1, 1, 1, 0] and shape(8192, 4096, 2, 4, 1, 2)[3] == 1


def test_columns_are_whole_tiles(rule):
    for R in (1, 64, 1000, 9000):
        for T in (1, 16, 17, 40, 64, 65, 500, 1030):
            for elem in (1, 2, 4):
                p = rule(R, 1024, 2, 4, T, elem)
                assert p["Tp"] >= T and p["Tp"] % (16 * p["nt"]) == 0 and p["Tp"] - T < 16 * p["nt"]
                assert (p["rg"], p["nt"]) in ((1, 1), (2, 2), (2, 4)) and (elem != 4 or p["nt"] < 4)


def test_gradient_is_cut_into_whole_steps(rule):
    for R, K, T in ((11008, 4096, 2048), (1000, 768, 333), (64, 64, 4000), (8000, 64, 1), (1, 64, 1)):
        p = rule(R, K, 2, 4, T, 2)
        assert 0 <= p["tile"] <= 2
        for splits, length in ((p["splits_x"], R), (p["splits_w"], T)):
            assert 1 <= splits <= 32 and (splits == 1 or -(-length // 64) // splits >= 4)
