// Beam search's selection: the num_out largest of
//   total(w, t) = scores[w] + logits[w][t] - log sum_u exp(logits[w][u])
// over a request's beams w and the vocabulary, equal ones by the lower w*V + t.
//
// Bound by HBM: the logits are read once. The first kernel streams them in
// units of 512 elements, a warp each, and leaves a unit's largest logit m and
// sum exp(x - m). A total grows with its logit, so the n largest elements lie in
// the n units with the largest maxima (an element of any other unit has n better
// ones in front of it, one in each of those). The second kernel, a CTA for each
// request, joins the units' sums into the rows' log sums, finds a bound that at
// least n units reach, reads those units again (some n KB) and sorts what passes
// the bound by the exact comparison: totals in 64 bits, then positions.
#include <math.h>

#include <atomic>

#include "block_common.h"
#include "common.cuh"
#include "moe_decode.h"
#include "vec_math.cuh"

namespace moe {
namespace {

constexpr int kUnit = 512;            // elements that a warp reduces at a time
constexpr int kThreads = 256;         // of the first kernel
constexpr int kJoinThreads = 1024;    // of the second
constexpr int kBests = 256;           // among them the bound is found, one of four threads each
constexpr int kList = 1024;           // candidates at hand
constexpr int kEach = kUnit / kWarp;  // elements of a unit for a lane
constexpr int kCached = 8192;         // units of a request that fit shared memory beside the list of those picked
constexpr float kLog2e = 1.4426950408889634f;

struct SelectArgs {
  const void* logits;
  int64_t row_stride;
  const float* scores;
  const uint8_t* ended;
  float2* units;  // [rows][units]: maximum and sum
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  int64_t vocab, requests;
  int32_t beams, per_row, num_out, end_token;  // per_row: units of a row
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The larger, or NaN where one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// A lane's part of a unit, as loaded.
template <typename ET, int VB> struct Part {
  using V = typename Vec<VB>::T;
  static constexpr int kElems = VB / Elem<ET>::kBytes, kVecs = kEach / kElems;
  V v[kVecs];
  __device__ __forceinline__ void load(const void* row, int first, int lane) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = ld_stream(reinterpret_cast<const V*>(static_cast<const char*>(row) + (int64_t)first * Elem<ET>::kBytes) + i * kWarp + lane);
  }
};

template <typename ET, int VB>
__global__ void __launch_bounds__(kThreads) select_units_kernel(const SelectArgs a) {
  using P = Part<ET, VB>;
  using E1 = typename Vec<Elem<ET>::kBytes>::T;
  constexpr bool kPairs = VB >= 4 && Elem<ET>::kBytes == 2;
  await_previous_kernel();
  const int lane = lane_id(), C = a.per_row;
  const int64_t total = a.requests * a.beams * C, warps = (int64_t)gridDim.x * (kThreads / kWarp);
  const int64_t rows_on = warps / C;
  const int units_on = (int)(warps - rows_on * C);
  int64_t u = (int64_t)blockIdx.x * (kThreads / kWarp) + threadIdx.x / kWarp;
  int64_t row = u / C;
  int c = (int)(u - row * C);
  const auto at = [&](int64_t r) { return static_cast<const char*>(a.logits) + r * a.row_stride * Elem<ET>::kBytes; };
  const auto full = [&](int unit) { return (int64_t)(unit + 1) * kUnit <= a.vocab; };
  P next;
  if (u < total && full(c)) next.load(at(row), c * kUnit, lane);
  for (; u < total; u += warps) {
    const int64_t row_now = row;
    const int c_now = c;
    P part = next;
    row += rows_on;
    c += units_on;
    if (c >= C) {
      c -= C;
      ++row;
    }
    if (u + warps < total && full(c)) next.load(at(row), c * kUnit, lane);  // on its way while this one is reduced
    if (a.ended != nullptr && a.ended[row_now]) continue;
    if (!full(c_now)) {  // the row's last unit, element by element
      const E1* p = reinterpret_cast<const E1*>(at(row_now)) + (int64_t)c_now * kUnit;
      const int n = (int)(a.vocab - (int64_t)c_now * kUnit);
      float x[kEach], m = -INFINITY;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        x[i] = i * kWarp + lane < n ? Lanes<Elem<ET>::kBytes, ET>::get(ld_stream(p + i * kWarp + lane), 0) : -INFINITY;
        m = max_nan(m, x[i]);
      }
#pragma unroll
      for (int d = 1; d < kWarp; d <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
      const float base = m == -INFINITY ? 0.0f : m;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kEach; ++i) sum += ex2((x[i] - base) * kLog2e);
#pragma unroll
      for (int d = 1; d < kWarp; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) a.units[u] = make_float2(m, sum);
      continue;
    }
    float m;
    if constexpr (kPairs) {
      uint32_t top = Words<typename P::V>::get(part.v[0], 0);
#pragma unroll
      for (int i = 0; i < P::kVecs; ++i)
#pragma unroll
        for (int q = 0; q < Words<typename P::V>::N; ++q) top = max_nan_bf16x2(top, Words<typename P::V>::get(part.v[i], q));
      m = max_nan(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u));
    } else {
      m = Lanes<VB, ET>::get(part.v[0], 0);
#pragma unroll
      for (int i = 0; i < P::kVecs; ++i)
#pragma unroll
        for (int q = 0; q < P::kElems; ++q) m = max_nan(m, Lanes<VB, ET>::get(part.v[i], q));
    }
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float base = m == -INFINITY ? 0.0f : m;
    // The difference first: its rounding is the element's own, where one of m * log2 e would be the whole unit's.
    const uint64_t minus = f2_pack(__float_as_uint(-base), __float_as_uint(-base)), log2e = f2_pack(__float_as_uint(kLog2e), __float_as_uint(kLog2e));
    uint64_t sums[2] = {0, 0};
    const auto add = [&](float x0, float x1, int k) {
      const uint64_t d = f2_mul(f2_add(f2_pack(__float_as_uint(x0), __float_as_uint(x1)), minus), log2e);
      float d0, d1;
      f2_unpack(d, d0, d1);
      sums[k & 1] = f2_add(sums[k & 1], f2_pack(__float_as_uint(ex2(d0)), __float_as_uint(ex2(d1))));
    };
    if constexpr (P::kElems >= 2) {
#pragma unroll
      for (int i = 0; i < P::kVecs; ++i)
#pragma unroll
        for (int q = 0; q < P::kElems; q += 2) add(Lanes<VB, ET>::get(part.v[i], q), Lanes<VB, ET>::get(part.v[i], q + 1), i + q / 2);
    } else {
#pragma unroll
      for (int i = 0; i < P::kVecs; i += 2) add(Lanes<VB, ET>::get(part.v[i], 0), Lanes<VB, ET>::get(part.v[i + 1], 0), i / 2);
    }
    float s0, s1;
    f2_unpack(f2_add(sums[0], sums[1]), s0, s1);
    float sum = s0 + s1;
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) a.units[u] = make_float2(m, sum);
  }
}

// Orders as its double does, NaN excluded.
__device__ __forceinline__ uint64_t key_of(double v) {
  const int64_t b = __double_as_longlong(v + 0.0);  // -0.0 as +0.0
  return (uint64_t)(b ^ ((b >> 63) | INT64_MIN));
}
__device__ __forceinline__ double value_of(uint64_t k) {
  const int64_t b = (int64_t)k;
  return __longlong_as_double(b < 0 ? b ^ INT64_MIN : ~b);
}
__device__ __forceinline__ bool better(uint64_t ka, uint32_t ia, uint64_t kb, uint32_t ib) {
  return ka > kb || (ka == kb && ia < ib);
}

// Sorts the list's first `n` (best first), with what lies behind up to the next power of two as the worst.
__device__ __forceinline__ void sort_list(uint64_t* keys, uint32_t* at, int n) {
  int size = 2;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += kJoinThreads) {
    keys[i] = 0;
    at[i] = 0xffffffffu;
  }
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kJoinThreads) {
        const int lo = (i / j) * 2 * j + i % j, hi = lo + j;
        const uint64_t ka = keys[lo], kb = keys[hi];
        const uint32_t ia = at[lo], ib = at[hi];
        if (better(kb, ib, ka, ia) == ((lo & k) == 0)) {
          keys[lo] = kb;
          keys[hi] = ka;
          at[lo] = ib;
          at[hi] = ia;
        }
      }
      __syncthreads();
    }
}

// What a total may be at least and at most when x + shift is t in 32 bits: the
// shift (of a score, a maximum and a logarithm whose sizes add up to `size`)
// and the sum are each off by 2^-23 of their size at most.
__device__ __forceinline__ float slack(float t, float size) { return 3e-7f * (fabsf(t) + size); }

template <typename ET>
__global__ void __launch_bounds__(kJoinThreads) select_join_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint64_t s_keys[kList];
  __shared__ uint32_t s_at[kList];
  __shared__ float s_x[kList];
  __shared__ double s_log[MOE_BEAM_MAX_BEAMS];  // of the row's sum exp(x - maximum)
  __shared__ float2 s_sum[MOE_BEAM_MAX_BEAMS];
  __shared__ float s_max[MOE_BEAM_MAX_BEAMS], s_score[MOE_BEAM_MAX_BEAMS];
  __shared__ float s_shift[MOE_BEAM_MAX_BEAMS], s_size[MOE_BEAM_MAX_BEAMS];  // total - logit, rounded; NaN: no candidates
  __shared__ __align__(16) float s_best[kBests];
  __shared__ float s_bound;
  __shared__ int s_picked, s_count, s_more;
  await_previous_kernel();
  const int lane = lane_id(), warp = threadIdx.x / kWarp, n = a.num_out, C = a.per_row, all = a.beams * C;
  const int64_t row0 = (int64_t)blockIdx.x * a.beams;
  int* picks = reinterpret_cast<int*>(smem);  // units that reach the bound
  const float2* units = a.units + row0 * C;
  if (threadIdx.x < a.beams) s_score[threadIdx.x] = a.scores[row0 + threadIdx.x];
  if (all <= kCached) {
    float2* own = reinterpret_cast<float2*>(smem + (size_t)(all + 1) / 2 * 8);
    for (int i = threadIdx.x; i < all; i += kJoinThreads) own[i] = units[i];
    units = own;
  }
  if (threadIdx.x == 0) {
    s_picked = s_count = s_more = 0;
    s_bound = -INFINITY;
  }
  __syncthreads();
  for (int w = warp; w < a.beams; w += kJoinThreads / kWarp) {
    float m = -INFINITY;
    for (int i = lane; i < C; i += kWarp) m = fmaxf(m, units[w * C + i].x);
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float sum = 0.0f, rest = 0.0f, e;  // sum + rest: the GPU has few 64-bit units
    for (int i = lane; i < C; i += kWarp) {
      const float2 u = units[w * C + i];
      if (u.x == -INFINITY && u.y == u.y) continue;
      two_sum(sum, u.y * ex2((u.x - m) * kLog2e), sum, e);
      rest += e;
    }
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) {
      const float other = __shfl_xor_sync(0xffffffffu, sum, d);
      rest += __shfl_xor_sync(0xffffffffu, rest, d);
      two_sum(sum, other, sum, e);
      rest += e;
    }
    if (lane == 0) {
      const float score = s_score[w], log_sum = logf(sum);
      const bool ended = a.ended != nullptr && a.ended[row0 + w];
      const float shift = (score - m) - log_sum;
      s_max[w] = m;
      s_sum[w] = make_float2(sum, rest);
      s_shift[w] = !ended && isfinite(m) && isfinite(log_sum) && isfinite(score) ? shift : NAN;
      s_size[w] = fabsf(score) + fabsf(m) + fabsf(log_sum);
      if (ended && isfinite(score)) {
        const int at = atomicAdd(&s_count, 1);
        s_x[at] = score;
        s_at[at] = (uint32_t)(w * a.vocab + a.end_token);
      }
    }
  }
  __syncthreads();
  // The rows' logarithms, for the totals in 64 bits, by one warp while the others go on.
  if (warp == kJoinThreads / kWarp - 1)
    for (int w = lane; w < a.beams; w += kWarp) s_log[w] = log((double)s_sum[w].x + (double)s_sum[w].y);
  // A bound that n units reach: the n-th of kBests sets' best ones, in 32 bits.
  float best = -INFINITY;
  for (int i = threadIdx.x; i < all; i += kJoinThreads) {
    const int w = i / C;
    const float t = units[i].x + s_shift[w];
    best = fmaxf(best, t - slack(t, s_size[w]));  // NaN leaves best as it is
  }
  best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
  best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
  const int mine = threadIdx.x / 4, quarter = threadIdx.x & 3;
  if (quarter == 0) s_best[mine] = best;
  __syncthreads();
  int rank = 0;
#pragma unroll 4
  for (int i = quarter; i < kBests / 4; i += 4) {
    const float4 o = reinterpret_cast<const float4*>(s_best)[i];
    rank += (o.x > best || (o.x == best && 4 * i < mine)) + (o.y > best || (o.y == best && 4 * i + 1 < mine)) +
            (o.z > best || (o.z == best && 4 * i + 2 < mine)) + (o.w > best || (o.w == best && 4 * i + 3 < mine));
  }
  rank += __shfl_xor_sync(0xffffffffu, rank, 1);
  rank += __shfl_xor_sync(0xffffffffu, rank, 2);
  if (rank == n - 1 && quarter == 0) s_bound = best;
  __syncthreads();
  float bound = s_bound;
  const auto passes = [&](float x, float shift, float size) {
    const float t = x + shift;
    return x > -INFINITY && t + slack(t, size) >= bound;  // false for a NaN shift
  };
  for (int i = threadIdx.x; i < all; i += kJoinThreads) {
    const int w = i / C;
    if (passes(units[i].x, s_shift[w], s_size[w])) picks[atomicAdd(&s_picked, 1)] = i;
  }
  __syncthreads();
  // Entries of the list from `done` on get their keys.
  int done = 0;
  const auto keys_to = [&](int count) {
    for (int i = done + threadIdx.x; i < count; i += kJoinThreads) {
      const int w = (int)(s_at[i] / a.vocab);
      // The maximum off first: a row of a type's lowest value has a log sum that 64 bits lose beside it.
      s_keys[i] = s_shift[w] == s_shift[w] ? key_of((double)s_score[w] + (((double)s_x[i] - (double)s_max[w]) - s_log[w]))
                                           : key_of((double)s_x[i]);  // a beam at its end: its score
    }
    done = count;
    __syncthreads();
  };
  const int picked = s_picked;
  for (int p0 = 0; p0 < picked; p0 += kJoinThreads / kWarp) {
    const int u = p0 + warp < picked ? picks[p0 + warp] : -1;
    const int w = u < 0 ? 0 : u / C, first = (u < 0 ? 0 : u - w * C) * kUnit;
    const float shift = s_shift[w], size = s_size[w];
    const auto* row = reinterpret_cast<const typename Vec<Elem<ET>::kBytes>::T*>(
        static_cast<const char*>(a.logits) + (row0 + w) * a.row_stride * Elem<ET>::kBytes);
    float x[kEach];
    unsigned pass = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int t = first + j * kWarp + lane;
      x[j] = u >= 0 && t < a.vocab ? Lanes<Elem<ET>::kBytes, ET>::get(ld_stream(row + t), 0) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) pass |= (passes(x[j], shift, size) ? 1u : 0u) << j;
    const auto add = [&](int j) {
      const int at = atomicAdd(&s_count, 1);
      s_x[at] = x[j];
      s_at[at] = (uint32_t)(w * a.vocab + first + j * kWarp + lane);
    };
    const int more = __reduce_add_sync(0xffffffffu, __popc(pass));
    if (lane == 0 && more > 0) atomicAdd(&s_more, more);
    __syncthreads();
    const bool room = s_count + s_more <= kList;
    __syncthreads();
    if (threadIdx.x == 0) s_more = 0;  // the next round adds to it behind the barrier below
    if (room) {
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (pass >> j & 1) add(j);
      __syncthreads();
      continue;
    }
    // One element of each lane of half a warp of them at a time, the list cut to the best n in between.
    for (int j2 = 0; j2 < 2 * kEach; ++j2) {
      __syncthreads();
      const int have = s_count;
      __syncthreads();
      if (have > kList - kJoinThreads / 2) {
        keys_to(have);
        sort_list(s_keys, s_at, have);
        if (have >= n) bound = fmaxf(bound, __double2float_rd(value_of(s_keys[n - 1])));
        done = min(have, n);
        if (threadIdx.x == 0) s_count = done;
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (j == j2 / 2 && (warp & 1) == (j2 & 1) && (pass >> j & 1) && passes(x[j], shift, size)) add(j);
    }
    __syncthreads();
  }
  const int count = s_count;
  keys_to(count);
  const auto put = [&](int i, int to) {
    const int64_t o = (int64_t)blockIdx.x * n + to;
    const int64_t w = i >= 0 ? s_at[i] / a.vocab : 0;
    a.out_scores[o] = i >= 0 ? (float)value_of(s_keys[i]) : -INFINITY;
    a.out_parents[o] = i >= 0 ? (int32_t)(row0 + w) : -1;
    a.out_tokens[o] = i >= 0 ? (int32_t)(s_at[i] - w * a.vocab) : -1;
  };
  if (count <= kBests) {  // an entry's place is the number of better ones; four threads count for one
    int place = 0;
    if (mine < count) {
      const uint64_t key = s_keys[mine];
      const uint32_t at = s_at[mine];
      for (int i = quarter; i < count; i += 4) place += better(s_keys[i], s_at[i], key, at);
    }
    place += __shfl_xor_sync(0xffffffffu, place, 1);
    place += __shfl_xor_sync(0xffffffffu, place, 2);
    if (quarter == 0 && mine < count && place < n) put(mine, place);
  } else {
    sort_list(s_keys, s_at, count);
    if (threadIdx.x < n) put(threadIdx.x, threadIdx.x);
  }
  if (threadIdx.x < n && (int)threadIdx.x >= count) put(-1, threadIdx.x);
}

template <typename ET> int run_select(const SelectArgs& a, cudaStream_t s) {
  const int64_t units = a.requests * a.beams * a.per_row;
  const void* ptrs[1] = {a.logits};
  const int64_t stride = a.requests * a.beams > 1 ? a.row_stride * Elem<ET>::kBytes : 0;
  const int vb = pick_vec_bytes(stride, ptrs, 1, Elem<ET>::kBytes);
  const auto go = [&](auto k) {
    launch(k, persistent_grid(k, kThreads, 0, (units + kThreads / kWarp - 1) / (kThreads / kWarp)), kThreads, 0, s, a);
  };
  if (vb == 16) go(select_units_kernel<ET, 16>);
  else if (vb == 8) go(select_units_kernel<ET, 8>);
  else if (vb == 4) go(select_units_kernel<ET, 4>);
  else if constexpr (Elem<ET>::kBytes == 2) go(select_units_kernel<ET, 2>);
  const int rc = check_launch();
  if (rc != MOE_OK) return rc;
  static std::atomic<bool> raised[kSmemDevices];
  if (!allow_smem(select_join_kernel<ET>, raised)) return MOE_ERR_CUDA;
  const size_t all = (size_t)a.beams * a.per_row;
  launch(select_join_kernel<ET>, dim3((unsigned)a.requests), dim3(kJoinThreads), (all + 1) / 2 * 8 + (all <= kCached ? 8 * all : 0), s, a);
  return check_launch();
}

bool select_ok(int64_t num_requests, int32_t num_beams, int64_t vocab) { return num_requests >= 0 && num_beams >= 1 && vocab >= 1; }
bool select_supported(int64_t num_requests, int32_t num_beams, int64_t vocab) {
  // The last: the second kernel keeps a list of units in shared memory.
  return num_beams <= MOE_BEAM_MAX_BEAMS && vocab <= INT32_MAX && num_beams * vocab <= INT32_MAX &&
         num_requests * num_beams <= INT32_MAX && num_beams * ((vocab + kUnit - 1) / kUnit) <= MOE_BEAM_MAX_UNITS;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_beam_select_workspace_size(int64_t num_requests, int32_t num_beams, int64_t vocab) {
  if (!select_ok(num_requests, num_beams, vocab) || !select_supported(num_requests, num_beams, vocab)) return 0;
  const size_t units = (size_t)num_requests * num_beams * ((vocab + kUnit - 1) / kUnit);
  return units * sizeof(float2) + 16;
}

extern "C" int moe_beam_select(const void* logits, int32_t dtype, int64_t row_stride, const float* scores,
                               const uint8_t* ended, int64_t num_requests, int32_t num_beams, int64_t vocab,
                               int32_t num_out, int32_t end_token, float* out_scores, int32_t* out_parents,
                               int32_t* out_tokens, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  const int eb = dtype_bytes(dtype);
  if (!select_ok(num_requests, num_beams, vocab) || num_out < 1) return MOE_ERR_INVALID_ARG;
  if (num_requests * num_beams > 1 && row_stride < vocab) return MOE_ERR_INVALID_ARG;
  if (ended != nullptr && (end_token < 0 || end_token >= vocab)) return MOE_ERR_INVALID_ARG;
  if (eb == 0 || num_out > MOE_BEAM_MAX_OUT || !select_supported(num_requests, num_beams, vocab)) return MOE_ERR_UNSUPPORTED;
  if (num_requests == 0) return MOE_OK;
  if (logits == nullptr || scores == nullptr || out_scores == nullptr || out_parents == nullptr || out_tokens == nullptr ||
      workspace == nullptr || workspace_bytes < moe_beam_select_workspace_size(num_requests, num_beams, vocab))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, eb) || !aligned(scores, 4) || !aligned(out_scores, 4) || !aligned(out_parents, 4) ||
      !aligned(out_tokens, 4) || !aligned(workspace, 16))
    return MOE_ERR_UNSUPPORTED;
  SelectArgs a = {};
  a.logits = logits;
  a.row_stride = row_stride;
  a.scores = scores;
  a.ended = ended;
  a.units = static_cast<float2*>(workspace);
  a.out_scores = out_scores;
  a.out_parents = out_parents;
  a.out_tokens = out_tokens;
  a.vocab = vocab;
  a.requests = num_requests;
  a.beams = num_beams;
  a.per_row = (int32_t)((vocab + kUnit - 1) / kUnit);
  a.num_out = num_out;
  a.end_token = end_token;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == MOE_F32 ? run_select<float>(a, s) : run_select<__nv_bfloat16>(a, s);
}
