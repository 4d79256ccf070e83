// What the decode attention's kernels share: the arguments, the line of tiles and
// the warps' ranges of it, the rows' places, asynchronous copies.
#pragma once

#include <math.h>

#include <atomic>

#include "block_common.h"
#include "bulk.cuh"
#include "common.cuh"
#include "divisor.h"
#include "moe_decode.h"

namespace moe {

constexpr int kTile = 16;      // tokens of a tile, the unit of the ranges
constexpr int kMostWarps = 16; // of an SM, which has one CTA
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttendArgs {
  char* k;  // the cache; strides in bytes
  char* v;
  int64_t page_stride, token_stride, head_stride;
  const char* q;
  const char* k_new;  // nullptr: the new token is in the cache already
  const char* v_new;
  int64_t q_row, q_head, kn_row, kn_head, vn_row, vn_head;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lengths;
  void* out;
  float* lse;
  float* part_o;  // [slots][heads][D], not yet divided by the sum
  float2* part_ml;  // [slots][heads]: maximum in units of log 2, and sum
  int32_t* status;
  Divisor page;
  int64_t num_pages, window;
  int32_t seqs, heads, kv_heads, group, D;
  int32_t parts;       // pieces of a group, of kHeads query heads each
  int32_t ranges;      // at most
  int32_t max_tokens;  // table width * page size
  float scale;         // times log2 e
};

// The positions of sequence b that are looked at: [first, n).
__device__ __forceinline__ void span_of(const AttendArgs& a, int b, int& first, int& n) {
  n = a.lengths[b];
  n = n < 0 ? 0 : (n > a.max_tokens ? a.max_tokens : n);
  first = a.window > 0 && n > a.window ? n - (int)a.window : 0;
}
__device__ __forceinline__ int tiles_of(const AttendArgs& a, int b) {
  int first, n;
  span_of(a, b, first, n);
  return (n - first + kTile - 1) / kTile;
}
__device__ __forceinline__ int ranges_of(const AttendArgs& a, int total) {  // total > 0
  return total < a.ranges ? total : a.ranges;
}
__device__ __forceinline__ int range_begin(int r, int ranges, int total) { return (int)((int64_t)r * total / ranges); }
// The range that tile x lies in: the last r whose begin is not behind x.
__device__ __forceinline__ int range_at(int x, int ranges, int total) {
  return (int)((((int64_t)x + 1) * ranges - 1) / total);
}

// Sum over the CTA of v, and in `before` the sum over the threads in front.
__device__ __forceinline__ int block_prefix(int v, int* s_warp, int& before) {
  const int lane = lane_id(), warp = threadIdx.x / kWarp, warps = blockDim.x / kWarp;
  int x = v;
#pragma unroll
  for (int d = 1; d < kWarp; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += o;
  }
  if (lane == kWarp - 1) s_warp[warp] = x;
  __syncthreads();
  int sum = 0, total = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) sum += s_warp[w];
    total += s_warp[w];
  }
  before = sum + x - v;
  return total;
}

// Where a warp is in the line of tiles.
struct Cursor {
  int b, tile, tiles, first, n;
  // The new token's position, or -1. A length beyond the table has no place for it: the last
  // position that there is holds a token already, in a page that other sequences may share.
  int fresh;
  __device__ __forceinline__ void enter(const AttendArgs& a) {
    span_of(a, b, first, n);
    tiles = (n - first + kTile - 1) / kTile;
    fresh = a.k_new != nullptr && a.lengths[b] <= a.max_tokens ? n - 1 : -1;
  }
  // Its row of the tile; outside [0, kTile): the tile has none.
  __device__ __forceinline__ int fresh_row() const { return fresh - (first + tile * kTile); }
  // There is a next tile. (The bounds on b keep the steps inside the table should lengths change meanwhile.)
  __device__ __forceinline__ void next(const AttendArgs& a) {
    if (++tile < tiles) return;
    tile = 0;
    do {
      if (b < a.seqs - 1) ++b;
      enter(a);
    } while (tiles == 0 && b < a.seqs - 1);
  }
};

// From a maximum (in units of log 2) and a sum: what the sums are multiplied by, and
// the log sum. A row without positions has sum 0; a NaN stays one.
__device__ __forceinline__ float share_of(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }
__device__ __forceinline__ float log_sum_of(float m, float sum) { return sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2; }

// The joining kernel may start: it waits for this one before it reads what it left.
__device__ __forceinline__ void start_next_kernel() { asm volatile("griddepcontrol.launch_dependents;"); }

__device__ __forceinline__ void check_length(const AttendArgs& a, int n) {
  if (blockIdx.x == 0 && (n < 0 || n > a.max_tokens)) flag_status(a.status, MOE_STATUS_BAD_INDEX);
}

// The tiles in front of the sequences of each thread, in prefix, and their sum.
__device__ __forceinline__ int line_prefix(const AttendArgs& a, int* prefix, int* s_warp) {
  const int t = threadIdx.x, chunk = (a.seqs + blockDim.x - 1) / blockDim.x;
  int mine = 0;
  for (int b = t * chunk; b < a.seqs && b < (t + 1) * chunk; ++b) {
    check_length(a, a.lengths[b]);
    mine += tiles_of(a, b);
  }
  int before;
  const int total = block_prefix(mine, s_warp, before);
  prefix[t] = before;
  __syncthreads();
  return total;
}
__device__ __forceinline__ Cursor find_tile(const AttendArgs& a, const int* prefix, int x) {
  const int chunk = (a.seqs + blockDim.x - 1) / blockDim.x;
  int lo = 0, hi = blockDim.x;  // the last thread with prefix <= x
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (prefix[mid] <= x) lo = mid; else hi = mid;
  }
  Cursor c;
  c.b = lo * chunk;
  c.tile = x - prefix[lo];
  c.enter(a);
  while (c.tile >= c.tiles && c.b < a.seqs - 1) {
    c.tile -= c.tiles;
    ++c.b;
    c.enter(a);
  }
  return c;
}

// Where the keys of a tile are: each of the lanes 0 to 15 answers for one
// position, with its page's number and then its offset in bytes (-1: absent).
__device__ __forceinline__ int page_entry(const AttendArgs& a, const Cursor& c, int row) {
  const int pos = c.first + c.tile * kTile + row;
  return pos < c.n ? a.table[c.b * a.table_stride + a.page.of(pos)] : -1;
}
__device__ __forceinline__ int64_t row_offset(const AttendArgs& a, const Cursor& c, int row, int page, int kv) {
  const int pos = c.first + c.tile * kTile + row;
  if (pos >= c.n) return -1;
  if (page < 0 || page >= a.num_pages) {
    flag_status(a.status, MOE_STATUS_BAD_INDEX);
    return -1;
  }
  return page * a.page_stride + (pos - a.page.of(pos) * a.page.d) * a.token_stride + kv * a.head_stride;
}

// A warp's (or team's) range r of a head's line, and which piece hv of a group of heads.
struct Share {
  int r, hv;
};
__device__ __forceinline__ Share share_at(int unit, int pieces) { return {unit / pieces, unit % pieces}; }

// The share of worker `place` of the CTA's `workers`: how many tiles, and where
// the first is. Neighbouring workers take neighbouring heads of a range; where
// there are fewer tiles than ranges the CTAs take turns, so that every SM has some
// (one of 200 tokens, 32 heads of 128 on 8, bf16: 6.5 us instead of 6.7).
__device__ __forceinline__ int my_range(const AttendArgs& a, int place, int workers, int* prefix, int* s_warp, Share& share, Cursor& c) {
  const int pieces = a.kv_heads * a.parts;
  share = share_at(blockIdx.x * workers + place, pieces);
  const Share spread = share_at(place * gridDim.x + blockIdx.x, pieces);
  int total, before = 0, x = 0;  // x: tiles up to the lane's sequence
  const bool few = a.seqs <= kWarp;
  Cursor own = {lane_id(), 0, 0, 0, 0, -1};
  if (few) {  // every warp for itself
    if (own.b < a.seqs) {
      check_length(a, a.lengths[own.b]);
      own.enter(a);
    }
    x = own.tiles;
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, x, d);
      if (own.b >= d) x += o;
    }
    total = __shfl_sync(0xffffffffu, x, kWarp - 1);
  } else {
    total = line_prefix(a, prefix, s_warp);
  }
  if (total == 0) return 0;
  const int ranges = ranges_of(a, total);
  if (total < a.ranges) share = spread;
  const int r = share.r;
  if (r >= ranges) return 0;
  const int lo = range_begin(r, ranges, total), count = range_begin(r + 1, ranges, total) - lo;
  if (count <= 0) return 0;
  if (few) {
    c.b = __ffs(__ballot_sync(0xffffffffu, x > lo)) - 1;
    before = __shfl_sync(0xffffffffu, x - own.tiles, c.b);
    c.tile = lo - before;
    c.tiles = __shfl_sync(0xffffffffu, own.tiles, c.b);
    c.first = __shfl_sync(0xffffffffu, own.first, c.b);
    c.n = __shfl_sync(0xffffffffu, own.n, c.b);
    c.fresh = __shfl_sync(0xffffffffu, own.fresh, c.b);
  } else {
    c = find_tile(a, prefix, lo);
  }
  return count;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

template <int BYTES> __device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int bytes) {
  if constexpr (BYTES == 16) cp_async16(dst, src, bytes); else cp_async4(dst, src, bytes);
}

// Ranges of the line for a kernel of `warps` warps an SM that takes kHeads query heads at a time.
inline void cut(AttendArgs& a, int heads_at_once, int warps) {
  a.parts = (a.group + heads_at_once - 1) / heads_at_once;
  const int64_t r = (int64_t)num_sms() * warps / ((int64_t)a.kv_heads * a.parts);
  a.ranges = (int32_t)(r < 1 ? 1 : r);
}
inline unsigned ctas_of(const AttendArgs& a, int warps) {
  return (unsigned)(((int64_t)a.ranges * a.kv_heads * a.parts + warps - 1) / warps);
}

// The first kernels (they set a.parts and a.ranges, which the joining kernel needs too).
int attend_rows(AttendArgs& a, bool pieces, cudaStream_t s);  // fp32; pieces: rows of 16-byte pieces on 16 bytes
int attend_mma_16(AttendArgs& a, cudaStream_t s);  // bf16 rows of 16-byte pieces on 16 bytes, and
int attend_mma_4(AttendArgs& a, cudaStream_t s);   // rows of 4-byte words on 4; query rows and outputs on 4 for both
int attend_mma_2(AttendArgs& a, cudaStream_t s);   // any bf16 rows

}  // namespace moe
