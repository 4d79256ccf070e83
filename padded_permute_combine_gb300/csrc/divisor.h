// Division by numbers that a kernel is launched with.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// Quotients by a divisor known at launch, for numerators below 2^31: with
// s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1, n / d = (mulhi(n, m) + n) >> s
// (Granlund and Montgomery, Division by Invariant Integers, 1994).
struct Divisor {
  uint32_t d, m, s;
  Divisor() : Divisor(1) {}
  explicit Divisor(uint32_t by) : d(by), m(0), s(0) {
    while ((1ull << s) < by) ++s;
    m = (uint32_t)(((1ull << 32) * ((1ull << s) - by)) / by + 1);
  }
  __host__ __device__ uint32_t of(uint32_t n) const {
#ifdef __CUDA_ARCH__
    return (__umulhi(n, m) + n) >> s;
#else
    return ((uint32_t)((uint64_t)n * m >> 32) + n) >> s;
#endif
  }
};

}  // namespace moe
