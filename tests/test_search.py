"""csrc/search.h on the CPU: the place of the last number that is at most
another, in up to 2^31 - 1 of them, without a look outside."""
import os
import shutil
import subprocess

import pytest

from padded_permute_combine_gb300 import build as libbuild

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "search.h"
struct Steps {  // 0, 0, .., width, width, .., 2 width: `width` places a step
  int n, width;
  mutable int64_t outside = 0;
  int operator[](int i) const {
    if (i < 0 || i >= n) {
      ++outside;
      return 0;
    }
    return i / width * width;
  }
};
int main() {
  const int most = 0x7fffffff;
  int64_t bad = 0;
  for (int n : {1, 2, 3, 1000, (1 << 30) - 1, 1 << 30, (1 << 30) + 1, (1 << 30) + 12345, most - 1, most})
    for (int width : {1, 3, 1 << 20}) {
      const Steps s{n, width};
      for (int64_t t : {int64_t(-1), int64_t(0), int64_t(1), int64_t(n) / 2, int64_t(n) - 2, int64_t(n) - 1, int64_t(n), int64_t(most)}) {
        int64_t want = t < 0 ? 0 : (t / width + 1) * width - 1;
        if (want > n - 1) want = n - 1;
        if (moe::last_at_most(s, n, t) != want) ++bad;
      }
      bad += s.outside;
    }
  std::printf("%lld\n", (long long)bad);
  return bad != 0;
}
"""


def test_places(tmp_path):
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if cxx is None:
        pytest.skip("no C++ compiler")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(libbuild._nvcc()))), "include")
    (tmp_path / "check.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-O1", "-fwrapv", "-std=c++17", "-I", libbuild.CSRC, "-isystem", cuda, str(tmp_path / "check.cpp"), "-o",
                    str(tmp_path / "check")], check=True)
    assert subprocess.run([str(tmp_path / "check")], capture_output=True, text=True, check=True, timeout=60).stdout.strip() == "0"
