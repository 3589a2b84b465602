"""The sizes of lm_sizes.py run the tiles that they are there for (on the CPU: a small C++ program
compiled with g++ includes the header that the library takes its choices from)."""
import os
import shutil
import subprocess

import pytest
import torch

from tests.lm_sizes import ORTH, XENT

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "masking_sparse_gemm_amd", "csrc")
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")

PROGRAM = r"""
#include <cstdio>
#include "nm_tiles.h"
using namespace nm;

int main() {
  const char* names[] = {"256", "128", "narrow"};
  char op;
  long R, K, n;
  while (std::scanf(" %c %ld %ld %ld", &op, &R, &K, &n) == 4) {
    if (op == 'x') {  // V, K, T
      const XentGradCut cut(R, K, n);
      const long rows = cut.piece < R ? cut.piece : R;
      const int loss = pick_tile(R, n, pad64(K) / 64);
      const int prob = pick_tile(pad64(rows), pad64(n), pad64(K) / 64);
      const int dw = pick_tile(rows, K, pad64(n) / 64);
      const bool both = dw == kTile128 && cut.tile_x == kTile128;
      std::printf("%s %s %s %s %d %ld\n", names[loss], names[prob], both ? "both" : names[dw],
                  both ? "both" : names[cut.tile_x], cut.splits, (R + cut.piece - 1) / cut.piece);
    } else if (op == 'm') {  // R, K, T
      std::printf("%s\n", column_lds(R, K, n) ? "whole" : "slices");
    } else {  // R, K, one part or two
      const long rp = pad64(R), kp = pad64(K), mp = R > K ? kp : rp, sum = R > K ? rp : kp;
      const auto pick = [&](long rows, long cols, long k, bool lower) {
        return n == 1 ? pick_orth_tile(kOrthTiles, rows, cols, (int)(k / 64), lower)
                      : pick_orth_tile(kOrthSplitTiles, rows, cols, (int)(k / 64), lower);
      };
      std::printf("%d %d %d\n", pick(mp, mp, sum, true), pick(mp, mp, mp, true),
                  pick(rp, kp, mp, false));
    }
  }
}
"""


def answers(tmp_path, lines):
    src, exe = tmp_path / "tiles.cpp", tmp_path / "tiles"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-Wall", "-I", CSRC, str(src), "-o", str(exe)])
    out = subprocess.run([str(exe)], input="\n".join(lines), capture_output=True, text=True,
                         timeout=60, check=True).stdout
    return [tuple(int(x) if x.isdigit() else x for x in line.split()) for line in out.splitlines()]


def test_xent_sizes_take_their_tiles(tmp_path):
    got = answers(tmp_path, ["x %d %d %d" % size for size in XENT])
    want = [tuple(int(x) if str(x).isdigit() else x for x in w) for w in XENT.values()]
    assert dict(zip(XENT, got)) == dict(zip(XENT, want))
    for product, tiles in enumerate(({"256", "128", "narrow"},) * 2 +
                                    ({"256", "128", "narrow", "both"},) * 2):
        assert {w[product] for w in XENT.values()} == tiles
    # dX adds up over pieces and splits at once on every tile
    assert {w[3] for w in XENT.values() if w[4] > 1 and w[5] > 1} == {"256", "128", "narrow", "both"}


def test_orthogonalize_sizes_take_their_tiles(tmp_path):
    got = answers(tmp_path, ["o %d %d %d" % (R, K, 1 if dt == torch.bfloat16 else 2)
                             for R, K, dt in ORTH])
    assert dict(zip(ORTH, got)) == ORTH
    for tall in (False, True):
        one = [w for (R, K, dt), w in ORTH.items() if dt == torch.bfloat16 and (R > K) == tall]
        assert {128, 192, 256} <= {w[0] for w in one} and {128, 192, 256} <= {w[1] for w in one}
        assert {128, 192, 256} <= {w[2] for w in one}
        two = [w for (R, K, dt), w in ORTH.items() if dt != torch.bfloat16 and (R > K) == tall]
        assert (128, 128, 128) in two


# what measured faster: X's columns whole in LDS, or slices of them
MATVEC = {(4096, 4096, 1): "whole", (4096, 4096, 8): "whole", (8192, 2048, 8): "whole",
          (4096, 6144, 8): "whole", (1024, 7168, 8): "slices",
          (4608, 4096, 8): "slices", (8192, 4096, 8): "slices", (24576, 1024, 8): "slices",
          (11008, 4096, 7): "whole", (11008, 4096, 8): "slices", (16384, 8192, 2): "whole",
          (16384, 8192, 5): "slices", (4096, 4096, 9): "slices", (40, 40001, 1): "slices"}


def test_few_columns_go_the_faster_way(tmp_path):
    got = answers(tmp_path, ["m %d %d %d" % size for size in MATVEC])
    assert {size: a for size, (a,) in zip(MATVEC, got)} == MATVEC
