"""csrc/smem_limit.h on the CPU, against a fake of the CUDA runtime: host
threads that raise a kernel's limit on dynamic shared memory together leave it
at all that a CTA can have."""
import os
import shutil
import subprocess

import pytest

from padded_permute_combine_gb300 import build as libbuild

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <set>
#include <thread>
#include <vector>
#include "smem_limit.h"

constexpr int kOptIn = 232448, kStatic = 1200;
thread_local int device = 0;
std::mutex lock;
int limit[128], sets = 0, fails = 0;
std::set<int> values;
std::atomic<bool> raised[moe::kSmemDevices];
void kernel(int) {}
void (*between)() = nullptr;  // what another thread does between the first one's set and its record

extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = device, cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void* f) {
  if (f != reinterpret_cast<const void*>(kernel)) return cudaErrorInvalidDeviceFunction;
  a->sharedSizeBytes = kStatic;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr which, int) {
  if (which != cudaDevAttrMaxSharedMemoryPerBlockOptin) return cudaErrorInvalidValue;
  return *v = kOptIn, cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute which, int v) {
  if (fails > 0) return --fails, cudaErrorInvalidValue;
  if (which != cudaFuncAttributeMaxDynamicSharedMemorySize || v > kOptIn - kStatic) return cudaErrorInvalidValue;
  {
    std::lock_guard<std::mutex> held(lock);
    limit[device] = v;
    values.insert(v);
    ++sets;
  }
  if (between != nullptr) {
    void (*other)() = between;
    between = nullptr;
    other();
  }
  return cudaSuccess;
}
}

#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); std::exit(1); } } while (0)

int main() {
  fails = 1;
  CHECK(!moe::allow_smem(kernel, raised));  // refused, and not recorded as done
  between = [] { CHECK(moe::allow_smem(kernel, raised)); };
  CHECK(moe::allow_smem(kernel, raised));
  CHECK(limit[0] == kOptIn - kStatic && sets == 2);
  CHECK(moe::allow_smem(kernel, raised) && sets == 2);  // once set, no call again
  device = 1;  // another device has its own limit
  CHECK(moe::allow_smem(kernel, raised) && limit[1] == kOptIn - kStatic && sets == 3);
  std::vector<std::thread> threads;
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([] {
      for (device = 2; device < 64; ++device) CHECK(moe::allow_smem(kernel, raised) && limit[device] == kOptIn - kStatic);
      device = 100;  // beyond the record: set at every call
      CHECK(moe::allow_smem(kernel, raised) && limit[100] == kOptIn - kStatic);
    });
  for (auto& t : threads) t.join();
  CHECK(values.size() == 1);
  return 0;
}
"""


def test_threads_leave_the_whole_limit(tmp_path):
    gxx = shutil.which(os.environ.get("CXX", "g++"))
    if gxx is None:
        pytest.skip("g++ not found")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(libbuild._nvcc()))), "include")
    (tmp_path / "t.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "t")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", libbuild.CSRC, "-isystem", cuda, str(tmp_path / "t.cpp"),
                    "-o", exe, "-pthread"], check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stdout
