"""Which 16-byte pieces of a row the adapters' expand kernel loads (nm_piece.h),
checked on the host: the rule itself is compiled and run over every column count,
leading dimension and tile near the edges.

The kernel adds the low-rank term to rows of fp32 that are either the caller's Y
(the last row ends at column C: nothing after it belongs to Y) or a workspace of
whole pieces.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "structured_sparse_gemm_nm_amd", "csrc")

PROGRAM = r"""
#include "nm_piece.h"
#include <cstdio>
#include <initializer_list>

// Whole pieces of a tile: within `readable`, and each column that exists in its own piece.
static int check(int C, int64_t ldb, int64_t readable, int width, bool expect_whole) {
  int whole_tiles = 0;
  for (int c0 = 0; c0 < C; c0 += width) {
    if (!nm::whole_pieces(c0, width, C, ldb, readable)) continue;
    ++whole_tiles;
    if (ldb % 4) return printf("rows off 16 bytes: C %d ldb %ld\n", C, long(ldb));
    for (int c = c0; c < c0 + width; c += 4) {
      const int at = nm::piece_start(c, C);
      if (at % 4 || at + 4 > readable) return printf("past the row: C %d ldb %ld readable %ld c %d\n", C, long(ldb), long(readable), c);
      if (c < C && at != c) return printf("another piece: C %d c %d\n", C, c);
    }
  }
  if (expect_whole && whole_tiles != (C + width - 1) / width) return printf("slow tiles: C %d ldb %ld\n", C, long(ldb));
  return 0;
}

int main() {
  for (int width : {16, 64})
    for (int C = 1; C < 300; ++C) {
      for (int64_t ldb = C; ldb < C + 9; ++ldb)                      // Y itself
        if (check(C, ldb, C, width, ldb % 4 == 0 && C % 4 == 0)) return 1;
      const int64_t padded = (C + 3) / 4 * 4;                        // a workspace of whole pieces
      if (check(C, padded, padded, width, true)) return 1;
    }
  return 0;
}
"""


def test_no_piece_past_the_rows(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "pieces.cpp", tmp_path / "pieces"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stdout
