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

constexpr int kUnit = 512;        // elements that a warp reduces at a time
constexpr int kThreads = 256;
constexpr int kList = 1024;       // candidates at hand
constexpr int kEach = kUnit / kWarp;  // elements of a unit for a lane
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

template <typename ET, int VB>
__global__ void __launch_bounds__(kThreads) select_units_kernel(const SelectArgs a) {
  using V = typename Vec<VB>::T;
  using L = Lanes<VB, ET>;
  constexpr int kVecs = kUnit / (kWarp * L::kElems);  // of a lane
  await_previous_kernel();
  const int lane = lane_id();
  const int64_t total = a.requests * a.beams * a.per_row, warps = (int64_t)gridDim.x * (kThreads / kWarp);
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / kWarp) + threadIdx.x / kWarp; u < total; u += warps) {
    const int64_t row = u / a.per_row;
    const int first = (int)(u - row * a.per_row) * kUnit;
    if (a.ended != nullptr && a.ended[row]) continue;
    const char* at = static_cast<const char*>(a.logits) + (row * a.row_stride + first) * Elem<ET>::kBytes;
    const int n = (int)(a.vocab - first < kUnit ? a.vocab - first : kUnit);
    float x[kVecs * L::kElems];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = (i * kWarp + lane) * L::kElems;
      if (e + L::kElems <= n) {
        const V v = ld_stream(reinterpret_cast<const V*>(at) + i * kWarp + lane);
#pragma unroll
        for (int q = 0; q < L::kElems; ++q) x[i * L::kElems + q] = L::get(v, q);
      } else {
#pragma unroll
        for (int q = 0; q < L::kElems; ++q)
          x[i * L::kElems + q] = e + q < n ? Lanes<Elem<ET>::kBytes, ET>::get(
                                                 ld_stream(reinterpret_cast<const typename Vec<Elem<ET>::kBytes>::T*>(at) + e + q), 0)
                                           : -INFINITY;
      }
    }
    float m = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kVecs * L::kElems; ++i) {
      m = fmaxf(m, x[i]);
      nan |= x[i] != x[i];
    }
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float base = m == -INFINITY ? 0.0f : m;
    float sum = 0.0f;
    // The difference first: its rounding is the element's own, where one of m * log2 e would be the whole unit's.
#pragma unroll
    for (int i = 0; i < kVecs * L::kElems; ++i) sum += exp2f((x[i] - base) * kLog2e);
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (__any_sync(0xffffffffu, nan)) sum = NAN;
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
  for (int i = n + threadIdx.x; i < size; i += kThreads) {
    keys[i] = 0;
    at[i] = 0xffffffffu;
  }
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
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
// shift and the sum are each off by 2^-24 of their size at most.
__device__ __forceinline__ float slack(float t, float shift) { return 2e-7f * (fabsf(t) + 2.0f * fabsf(shift)); }

template <typename ET>
__global__ void __launch_bounds__(kThreads) select_join_kernel(const SelectArgs a) {
  extern __shared__ int s_units[];  // units that reach the bound, beams * per_row at most
  __shared__ uint64_t s_keys[kList];
  __shared__ uint32_t s_at[kList];
  __shared__ double s_log[MOE_BEAM_MAX_BEAMS];  // of the row's sum exp(x - maximum)
  __shared__ float2 s_sum[MOE_BEAM_MAX_BEAMS];
  __shared__ float s_max[MOE_BEAM_MAX_BEAMS];
  __shared__ float s_shift[MOE_BEAM_MAX_BEAMS];  // total - logit, rounded; NaN: no candidates
  __shared__ float s_best[kThreads];
  __shared__ float s_bound;
  __shared__ int s_picked, s_count, s_more;
  await_previous_kernel();
  const int lane = lane_id(), warp = threadIdx.x / kWarp, n = a.num_out, C = a.per_row;
  const int64_t row0 = (int64_t)blockIdx.x * a.beams;
  const float2* units = a.units + row0 * C;
  for (int w = warp; w < a.beams; w += kThreads / kWarp) {
    float m = -INFINITY;
    for (int i = lane; i < C; i += kWarp) m = fmaxf(m, units[w * C + i].x);
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float sum = 0.0f, rest = 0.0f, e;  // sum + rest: the GPU has few 64-bit units
    for (int i = lane; i < C; i += kWarp) {
      const float2 u = units[w * C + i];
      if (u.x == -INFINITY && u.y == u.y) continue;
      two_sum(sum, u.y * exp2f((u.x - m) * kLog2e), sum, e);
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
      s_max[w] = m;
      s_sum[w] = make_float2(sum, rest);
    }
  }
  if (threadIdx.x == 0) {
    s_picked = s_count = s_more = 0;
    s_bound = -INFINITY;
  }
  __syncthreads();
  if (threadIdx.x < a.beams) {  // the logarithms of all rows at once
    const int w = threadIdx.x;
    const float score = a.scores[row0 + w];
    const bool ended = a.ended != nullptr && a.ended[row0 + w];
    const double log_sum = log((double)s_sum[w].x + (double)s_sum[w].y), lse = (double)s_max[w] + log_sum;
    s_log[w] = log_sum;
    s_shift[w] = !ended && isfinite(lse) && isfinite(score) ? (float)((double)score - lse) : NAN;
    if (ended && isfinite(score)) {
      const int at = atomicAdd(&s_count, 1);
      s_keys[at] = key_of((double)score);
      s_at[at] = (uint32_t)(w * a.vocab + a.end_token);
    }
  }
  __syncthreads();
  // A bound that n units reach: the n-th of the threads' best ones, in 32 bits.
  const int all = a.beams * C;
  float best = -INFINITY;
  for (int i = threadIdx.x; i < all; i += kThreads) {
    const float shift = s_shift[i / C], t = units[i].x + shift;
    best = fmaxf(best, t - slack(t, shift));  // NaN leaves best as it is
  }
  s_best[threadIdx.x] = best;
  __syncthreads();
  int rank = 0;
  for (int i = 0; i < kThreads; ++i) {
    const float o = s_best[i];
    rank += o > best || (o == best && i < (int)threadIdx.x);
  }
  if (rank == n - 1) s_bound = best;
  __syncthreads();
  float bound = s_bound;
  const auto passes = [&](float x, float shift) {
    const float t = x + shift;
    return x > -INFINITY && t + slack(t, shift) >= bound;  // false for a NaN shift
  };
  for (int i = threadIdx.x; i < all; i += kThreads)
    if (passes(units[i].x, s_shift[i / C])) s_units[atomicAdd(&s_picked, 1)] = i;
  __syncthreads();
  const int picked = s_picked;
  for (int p0 = 0; p0 < picked; p0 += kThreads / kWarp) {
    const int u = p0 + warp < picked ? s_units[p0 + warp] : -1;
    const int w = u < 0 ? 0 : u / C, first = (u < 0 ? 0 : u - w * C) * kUnit;
    const float shift = s_shift[w], score = a.scores[row0 + w];
    const double log_sum = s_log[w], m = s_max[w];
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
    for (int j = 0; j < kEach; ++j) pass |= (passes(x[j], shift) ? 1u : 0u) << j;
    const auto add = [&](int j) {
      const int at = atomicAdd(&s_count, 1);
      // The maximum off first: a row of a type's lowest value has a log sum that 64 bits lose beside it.
      s_keys[at] = key_of((double)score + (((double)x[j] - m) - log_sum));
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
#pragma unroll
    for (int j = 0; j < kEach; ++j) {  // an element of every lane at a time, the list cut to the best n in between
      __syncthreads();
      const int have = s_count;
      __syncthreads();
      if (have > kList - kThreads) {
        sort_list(s_keys, s_at, have);
        if (have >= n) bound = fmaxf(bound, __double2float_rd(value_of(s_keys[n - 1])));
        if (threadIdx.x == 0) s_count = min(have, n);
        __syncthreads();
      }
      if ((pass >> j & 1) && passes(x[j], shift)) add(j);
    }
    __syncthreads();
  }
  const int count = s_count;
  sort_list(s_keys, s_at, count);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int64_t o = (int64_t)blockIdx.x * n + i;
    const bool some = i < count;
    const int64_t w = some ? s_at[i] / a.vocab : 0;
    a.out_scores[o] = some ? (float)value_of(s_keys[i]) : -INFINITY;
    a.out_parents[o] = some ? (int32_t)(row0 + w) : -1;
    a.out_tokens[o] = some ? (int32_t)(s_at[i] - w * a.vocab) : -1;
  }
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
  launch(select_join_kernel<ET>, dim3((unsigned)a.requests), dim3(kThreads), (size_t)4 * a.beams * a.per_row, s, a);
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
