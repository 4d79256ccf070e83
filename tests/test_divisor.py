"""csrc/divisor.h on the CPU: quotients by multiplication equal division, for
every divisor of the page sizes and table widths that kernels are launched with
and numerators up to 2^31 - 1, the ones next to multiples above all."""
import os
import shutil
import subprocess

import pytest

from padded_permute_combine_gb300 import build as libbuild

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "divisor.h"
int main() {
  const uint32_t last = 0x7fffffffu;
  uint64_t seed = 1, bad = 0;
  const auto check = [&](const moe::Divisor& by, uint64_t n) { if (n <= last && by.of((uint32_t)n) != (uint32_t)n / by.d) ++bad; };
  for (uint64_t i = 0; i < 300000; ++i) {
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    uint32_t d = i < 70000 ? (uint32_t)i + 1 : (uint32_t)(seed >> 33) >> (i % 31);
    if (i % 97 == 0) d = 1u << (i % 31);
    if (i % 101 == 0) d = last - (uint32_t)(i % 5);
    if (d == 0) d = 1;
    const moe::Divisor by(d);
    const uint64_t k = (seed >> 20) % (last / d + 1);
    for (uint64_t n : {uint64_t(0), uint64_t(1), k * d, k * d + d - 1, k * d - (k ? 1 : 0), uint64_t(last), uint64_t(last) - 1, seed >> 34}) check(by, n);
  }
  std::printf("%llu\n", (unsigned long long)bad);
  return bad != 0;
}
"""


def test_quotients(tmp_path):
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if cxx is None:
        pytest.skip("no C++ compiler")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(libbuild._nvcc()))), "include")
    (tmp_path / "check.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", libbuild.CSRC, "-isystem", cuda, str(tmp_path / "check.cpp"), "-o",
                    str(tmp_path / "check")], check=True)
    assert subprocess.run([str(tmp_path / "check")], capture_output=True, text=True, check=True).stdout.strip() == "0"
