"""The grid of kernels with a block per few rows: no line of it reaches the 2^32 threads that a
launch refuses, every block index is covered once, and an index times the rows of a block stays
in 32 bits (csrc/grid.hpp, compiled for the host)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "recommender_embedding_tables_amd", "csrc")
PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "grid.hpp"
int main(int n, char** a) {
  for (int i = 1; i < n; ++i) {
    const embtab::Grid g = embtab::fold_grid(atoll(a[i]));
    printf("%u %u\\n", g.x, g.y);
  }
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_folded_grids(tmp_path):
    (tmp_path / "grid.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "grid")
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(tmp_path / "grid.cpp"), "-o", exe],
                   check=True)
    # (distinct rows, rows of a block): 4 at widths above 128, up to 256 at a width of 4
    cases = [(r, k) for k in (4, 8, 16, 32, 64, 128, 256)
             for r in (1, k, k + 1, 1 << 23, 1 << 26, (1 << 26) + 1, 1 << 27, (1 << 30) + 7,
                       (1 << 32) - 2)]
    blocks = [-(-r // k) for r, k in cases]
    out = subprocess.run([exe, *map(str, blocks)], check=True, capture_output=True, text=True)
    for (rows, k), b, line in zip(cases, blocks, out.stdout.splitlines()):
        x, y = map(int, line.split())
        assert x * 256 < 1 << 32 and y < 1 << 16, (rows, k)
        assert x * y >= b and x * (y - 1) < b, (rows, k)
        assert x * y * k <= 1 << 32, (rows, k)
