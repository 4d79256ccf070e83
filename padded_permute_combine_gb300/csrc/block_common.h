// What the layer norm and the few-token layer share.
#pragma once

#include <atomic>

#include "common.cuh"
#include "smem_limit.h"

namespace moe {

// The waits that moe_test_block_waits makes give up.
constexpr uint32_t kGiveUpWeights = 1, kGiveUpTokens = 2, kGiveUpProducts = 4, kGiveUpSums = 8, kGiveUpRows = 16;
std::atomic<uint32_t>& test_give_up();

// a * b + c of two packed fp32 pairs.
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// persistent_grid, without the question about occupancy where every SM gets one CTA at most.
template <typename Kernel> int grid_for(Kernel k, int threads, size_t smem, int64_t work_ctas) {
  if (work_ctas <= num_sms()) return work_ctas < 1 ? 1 : (int)work_ctas;
  return persistent_grid(k, threads, smem, work_ctas);
}

}  // namespace moe
