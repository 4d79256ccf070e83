// Search in ascending numbers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// The place of the last of n ascending numbers that is at most t (0 where none is), n up
// to 2^31 - 1: two places may add up to more than 32 bits hold, their distance does not.
template <typename Numbers> __host__ __device__ __forceinline__ int last_at_most(const Numbers& numbers, int n, int64_t t) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (numbers[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace moe
