"""An expert's rows and the number of token tiles from offsets on the device
(nm_offsets.h), checked on the host: the rule itself is compiled and run over
every list of offsets, good and bad, of few experts and tokens."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "structured_sparse_gemm_nm_amd", "csrc")

PROGRAM = r"""
#include "nm_offsets.h"
#include <cstdio>

int main() {
  for (int T = 0; T <= 5; ++T)
    for (int a = -2; a <= 7; ++a)
      for (int b = -2; b <= 7; ++b) {
        const int lo = nm::rows_lo(a, T), hi = nm::rows_hi(b, lo, T);
        if (lo < 0 || hi < lo || hi > T) return printf("outside: T %d offsets %d %d\n", T, a, b);
        if (a >= 0 && b >= a && b <= T && (lo != a || hi != b)) return printf("good offsets changed: %d %d\n", a, b);
      }
  // ascending offsets of three experts: their tiles never pass the bound, and reach it
  for (int BT = 1; BT <= 4; ++BT)
    for (int T = 0; T <= 9; ++T) {
      int64_t most = 0;
      for (int a = 0; a <= T; ++a)
        for (int b = a; b <= T; ++b) {
          const int n[3] = {a, b - a, T - b};
          int64_t tiles = 0;
          for (int e = 0; e < 3; ++e) tiles += (n[e] + BT - 1) / BT;
          if (tiles > most) most = tiles;
        }
      if (most != nm::group_max_tiles(T, 3, BT)) return printf("bound: T %d BT %d: %ld, not %ld\n", T, BT, long(most), long(nm::group_max_tiles(T, 3, BT)));
    }
  // every expert of the most given every token: the sum stops, and stays in range
  int sum = 0;
  for (int e = 0; e < 65535; ++e) {
    sum = nm::tile_sum(sum, 1 << 20);
    if (sum < 0 || sum > nm::kTileSumMax) return printf("overflow\n");
  }
  if (nm::tile_sum(nm::kTileSumMax, nm::kTileSumMax) != nm::kTileSumMax) return printf("overflow of two\n");
  if (nm::group_max_tiles(1 << 24, 65535, 16) >= nm::kTileSumMax) return printf("a tile's number passes the sums' end\n");
  return 0;
}
"""


def test_rows_and_tiles(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "offsets.cpp", tmp_path / "offsets"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout
