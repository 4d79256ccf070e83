// The turns of a warp over the units of rows.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// Rows of per_row units each, dealt to `warps` warps one after another: the unit that
// warp `first` is at. Up to 2^31 - 1 rows: the step behind the last of them, of up to
// `warps` rows, has to stay above them, which 31 bits would not hold.
struct UnitTurns {
  uint32_t row;
  int32_t c;  // unit of the row
  int32_t per_row, units_on;
  uint32_t rows_on;
  __host__ __device__ __forceinline__ UnitTurns(int first, int warps, int units_a_row)
      : row((uint32_t)(first / units_a_row)), c(first % units_a_row), per_row(units_a_row), units_on(warps % units_a_row), rows_on((uint32_t)(warps / units_a_row)) {}
  __host__ __device__ __forceinline__ void next() {
    row += rows_on;
    c += units_on;
    if (c >= per_row) {
      c -= per_row;
      ++row;
    }
  }
};

}  // namespace moe
