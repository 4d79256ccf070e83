// A kernel's limit on dynamic shared memory (host code alone).
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>

namespace moe {

constexpr int kSmemDevices = 64;

// Raises the limit, once per device, to all that a CTA can have beside the
// kernel's static part. Every call sets the same value, so host threads that
// come here together leave it at that, whoever is last. (Raised to what each
// call needs, it could end below what the record says: one thread sets 100 KB,
// another 60 KB, the first records 100 last, and calls of 80 KB then fail.)
template <typename Kernel> bool allow_smem(Kernel k, std::atomic<bool>* raised) {
  int dev = 0, most = 0;
  (void)cudaGetDevice(&dev);
  const bool recorded = dev >= 0 && dev < kSmemDevices;
  if (recorded && raised[dev].load(std::memory_order_relaxed)) return true;
  const void* f = reinterpret_cast<const void*>(k);
  cudaFuncAttributes own;
  if (cudaFuncGetAttributes(&own, f) != cudaSuccess ||
      cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
      cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)own.sharedSizeBytes) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  if (recorded) raised[dev].store(true, std::memory_order_relaxed);
  return true;
}

}  // namespace moe
