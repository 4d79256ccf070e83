"""csrc/unit_turns.h on the CPU: warps take every unit of up to 2^31 - 1 rows
once, and their step behind the last row leaves the rows."""
import os
import shutil
import subprocess

import pytest

from padded_permute_combine_gb300 import build as libbuild

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include <vector>
#include "unit_turns.h"
int main() {
  int64_t bad = 0;
  // Few units: each is taken once.
  for (int rows : {1, 7, 300})
    for (int per_row : {1, 2, 97})
      for (int warps : {8, 16, 4864}) {
        std::vector<int> seen((size_t)rows * per_row);
        for (int w = 0; w < warps; ++w)
          for (moe::UnitTurns t(w, warps, per_row); t.row < rows; t.next()) {
            if (t.c < 0 || t.c >= per_row) return 2;
            ++seen[(size_t)t.row * per_row + t.c];
          }
        for (int n : seen) bad += n != 1;
      }
  // As many rows as there may be, on the GPU's whole grid: no warp is anywhere else.
  for (int64_t rows : {(int64_t)0x7fffffff, (int64_t)0x7fffffff - 63, (int64_t)0x7fffffff - 4863})
    for (int per_row : {1, 3})
      for (int warps : {4736, 4864})
        for (int w : {0, 1, 1000, warps - 1}) {
          const int64_t units = rows * per_row, mine = (units - w + warps - 1) / warps;
          int64_t n = 0, at = w;
          moe::UnitTurns t(w, warps, per_row);
          for (; t.row < rows && n <= mine; t.next(), ++n, at += warps) bad += (int64_t)t.row * per_row + t.c != at;
          bad += n != mine;
        }
  std::printf("%lld\n", (long long)bad);
  return bad != 0;
}
"""


def test_turns(tmp_path):
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if cxx is None:
        pytest.skip("no C++ compiler")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(libbuild._nvcc()))), "include")
    (tmp_path / "check.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-O1", "-fwrapv", "-std=c++17", "-I", libbuild.CSRC, "-isystem", cuda, str(tmp_path / "check.cpp"), "-o",
                    str(tmp_path / "check")], check=True)
    assert subprocess.run([str(tmp_path / "check")], capture_output=True, text=True, check=True, timeout=120).stdout.strip() == "0"
