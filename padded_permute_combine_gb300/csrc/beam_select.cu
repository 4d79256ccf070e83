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
// the bound by the exact comparison: totals in some 48 bits, then positions.
#include <math.h>

#include <atomic>

#include "block_common.h"
#include "common.cuh"
#include "moe_decode.h"
#include "unit_turns.h"
#include "vec_math.cuh"

namespace moe {
namespace {

constexpr int kUnit = 512;            // elements that a warp reduces at a time
constexpr int kThreads = 256;         // of the first kernel
constexpr int kUnitCtas = 4;          // of it, on an SM
constexpr int kJoinThreads = 1024;    // of the second
constexpr int kBests = 256;           // most sets of units among whose best ones the bound is found
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
__global__ void __launch_bounds__(kThreads, kUnitCtas) select_units_kernel(const SelectArgs a) {
  using P = Part<ET, VB>;
  using E1 = typename Vec<Elem<ET>::kBytes>::T;
  constexpr bool kPairs = VB >= 4 && Elem<ET>::kBytes == 2;
  await_previous_kernel();
  const int lane = lane_id(), C = a.per_row, warps = (int)gridDim.x * (kThreads / kWarp);
  const uint32_t rows = (uint32_t)(a.requests * a.beams);
  const int whole = (int)(a.vocab / kUnit);  // units that are full
  UnitTurns turn((int)blockIdx.x * (kThreads / kWarp) + (int)threadIdx.x / kWarp, warps, C);
  const int64_t stride = a.row_stride * Elem<ET>::kBytes;
  const auto at = [&](uint32_t r, int unit) { return static_cast<const char*>(a.logits) + r * stride + (int64_t)unit * kUnit * Elem<ET>::kBytes; };
  P next;
  if (turn.row < rows && turn.c < whole) next.load(at(turn.row, turn.c), 0, lane);
  while (turn.row < rows) {
    const uint32_t row_now = turn.row;
    const int c_now = turn.c;
    P part = next;
    turn.next();
    if (turn.row < rows && turn.c < whole) next.load(at(turn.row, turn.c), 0, lane);  // on its way while this one is reduced
    if (a.ended != nullptr && a.ended[row_now]) continue;
    float2* const to = a.units + ((int64_t)row_now * C + c_now);
    if (c_now >= whole) {  // the row's last unit, element by element
      float x[kEach], m = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int64_t t = (int64_t)c_now * kUnit + i * kWarp + lane;
        x[i] = t < a.vocab ? Lanes<Elem<ET>::kBytes, ET>::get(ld_stream(reinterpret_cast<const E1*>(at(row_now, 0)) + t), 0) : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i) m = max_nan(m, x[i]);
#pragma unroll
      for (int d = 1; d < kWarp; d <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
      const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < kEach; ++i) sum += ex2((x[i] - base) * kLog2e);
#pragma unroll
      for (int d = 1; d < kWarp; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) *to = make_float2(m, sum);
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
    if (lane == 0) *to = make_float2(m, sum);
  }
}

// Numbers of some 48 bits as sums of two 32-bit ones, the second at most half
// a unit of the first's last place. (In 64-bit arithmetic, of which the GPU has
// little, the rows' logarithms alone took 3.7 us, and the candidates' totals 3.)
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair sum_of(float a, float b) {
  Pair p;
  two_sum(a, b, p.hi, p.lo);
  return p;
}
// log of s in [1, 2^100), off by 3e-9 at most: with s = 2^k f, f in [sqrt(1/2), sqrt(2)) and
// z = (f - 1) / (f + 1), log s = k log 2 + 2 z + 2 z^3 (1/3 + z^2/5 + ...), the first two terms in pairs.
__device__ __forceinline__ Pair log_of(Pair s) {
  int k = (int)(__float_as_uint(s.hi) >> 23) - 127;  // s.hi in 2^k [1, 2)
  if ((__float_as_uint(s.hi) & 0x7fffffu) > 0x3504f3u) ++k;
  const float down = __uint_as_float((uint32_t)(127 - k) << 23);
  const float f = s.hi * down, rest = s.lo * down;  // exact
  const float num = f - 1.0f, den = f + 1.0f, den_rest = f - (den - 1.0f) + rest;
  const float z = __fdiv_rn(num, den);
  const float z_rest = (fmaf(-z, den, num) + (rest - z * den_rest)) / den;
  const float w = z * z;
  const float cubic = 2.0f * z * w * fmaf(fmaf(fmaf(fmaf(1.0f / 11, w, 1.0f / 9), w, 1.0f / 7), w, 1.0f / 5), w, 1.0f / 3);
  constexpr float kHigh = 11356.0f / 16384, kLow = 3.194618495e-05f;  // of log 2: 14 bits, whose products with k are exact, and the rest
  const Pair p = sum_of((float)k * kHigh, 2.0f * z);
  return sum_of(p.hi, p.lo + fmaf((float)k, kLow, 2.0f * z_rest + cubic));
}
// score + ((x - m) - log_sum). The maximum goes off first: a row of a type's
// lowest value has a log sum that vanishes beside it.
__device__ __forceinline__ Pair total_of(float score, float x, float m, Pair log_sum) {
  const Pair d = sum_of(x, -m), t = sum_of(d.hi, -log_sum.hi), u = sum_of(score, t.hi);
  const Pair total = sum_of(u.hi, u.lo + (t.lo + (d.lo - log_sum.lo)));
  // Differences beyond 32 bits' range: a candidate all the same, behind every other.
  return fabsf(total.hi) < INFINITY && fabsf(total.lo) < INFINITY ? total : Pair{-3.0e38f, 0.0f};
}
// Orders as the pair does.
__device__ __forceinline__ uint32_t key_half(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0.0 as +0.0
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float half_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
__device__ __forceinline__ uint64_t key_of(Pair p) { return (uint64_t)key_half(p.hi) << 32 | key_half(p.lo); }
__device__ __forceinline__ Pair value_of(uint64_t k) { return {half_value((uint32_t)(k >> 32)), half_value((uint32_t)k)}; }
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

// The whole kernel is one request's, on one SM, and runs once: what counts is
// the number of instructions of all its warps, and the trips to memory.
template <typename ET, int VB>
__global__ void __launch_bounds__(kJoinThreads) select_join_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint64_t s_keys[kList];
  __shared__ uint32_t s_at[kList];
  __shared__ float s_x[kList];
  __shared__ Pair s_log[MOE_BEAM_MAX_BEAMS];  // of the row's sum exp(x - maximum)
  __shared__ float s_max[MOE_BEAM_MAX_BEAMS], s_score[MOE_BEAM_MAX_BEAMS];
  __shared__ float s_shift[MOE_BEAM_MAX_BEAMS], s_size[MOE_BEAM_MAX_BEAMS];  // total - logit, rounded; NaN: no candidates
  __shared__ __align__(16) uint32_t s_best[kBests];
  __shared__ uint32_t s_bound;
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
    s_bound = 0;
  }
  __syncthreads();
  for (int w = warp; w < a.beams; w += kJoinThreads / kWarp) {
    float m = -INFINITY;
#pragma unroll 4
    for (int i = lane; i < C; i += kWarp) m = fmaxf(m, units[w * C + i].x);
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float sum = 0.0f, rest = 0.0f, e;
#pragma unroll 4
    for (int i = lane; i < C; i += kWarp) {
      const float2 u = units[w * C + i];
      const bool none = u.x == -INFINITY && u.y == u.y;
      two_sum(sum, none ? 0.0f : u.y * ex2((u.x - m) * kLog2e), sum, e);
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
      const float score = s_score[w];
      const bool ended = a.ended != nullptr && a.ended[row0 + w];
      const bool finite = isfinite(m) && sum > 0.0f && sum < INFINITY && isfinite(score);
      const Pair log_sum = finite ? log_of(sum_of(sum, rest)) : Pair{0.0f, 0.0f};
      s_log[w] = log_sum;
      s_max[w] = m;
      s_shift[w] = !ended && finite ? (score - m) - log_sum.hi : NAN;
      s_size[w] = fabsf(score) + fabsf(m) + fabsf(log_sum.hi);
      if (ended && isfinite(score)) {
        const int at = atomicAdd(&s_count, 1);
        s_x[at] = score;
        s_at[at] = (uint32_t)(w * a.vocab + a.end_token);
      }
    }
  }
  __syncthreads();
  // A bound that n units reach: the n-th of the best ones of 128 sets of units
  // (256 for more than 32), as whole numbers that order as they do, cut to 24
  // bits, with the set's number below to keep them apart.
  const int group = n <= 32 ? 8 : 4, sets = kJoinThreads / group;  // threads of a set
  float best = -INFINITY;
  for (int i = threadIdx.x; i < all; i += kJoinThreads) {
    const int w = i / C;
    const float t = units[i].x + s_shift[w];
    best = fmaxf(best, t - slack(t, s_size[w]));  // NaN leaves best as it is
  }
  for (int d = 1; d < group; d <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, d));
  const int mine = threadIdx.x / group, member = threadIdx.x % group;
  const uint32_t key = (best > -INFINITY ? key_half(best) & ~255u : 0u) | (uint32_t)(sets - 1 - mine);
  if (member == 0) s_best[mine] = key;
  __syncthreads();
  int rank = 0;
  for (int i = member; i < sets / 4; i += group) {
    const uint4 o = reinterpret_cast<const uint4*>(s_best)[i];
    rank += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
  }
  for (int d = 1; d < group; d <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, d);
  if (rank == n - 1 && member == 0) s_bound = key & ~255u;
  __syncthreads();
  float bound = s_bound == 0 ? -INFINITY : half_value(s_bound);
  // The least logit of a row whose total may reach the bound; -infinity never does.
  const auto least = [&](int w) { return fmaxf((bound - s_shift[w]) - 6e-7f * (fabsf(bound) + s_size[w]), -3.4028235e38f); };
  for (int i = threadIdx.x; i < all; i += kJoinThreads) {
    const int w = i / C;
    if (s_shift[w] == s_shift[w] && units[i].x >= least(w)) picks[atomicAdd(&s_picked, 1)] = i;
  }
  __syncthreads();
  // Entries of the list from `done` on get their keys.
  int done = 0;
  const auto keys_to = [&](int count) {
    for (int i = done + threadIdx.x; i < count; i += kJoinThreads) {
      const int w = (int)(s_at[i] / (uint32_t)a.vocab);
      s_keys[i] = key_of(s_shift[w] == s_shift[w] ? total_of(s_score[w], s_x[i], s_max[w], s_log[w])
                                                  : Pair{s_x[i], 0.0f});  // a beam at its end: its score
    }
    done = count;
    __syncthreads();
  };
  const int picked = s_picked;
  for (int p0 = 0; p0 < picked; p0 += kJoinThreads / kWarp) {
    const int u = p0 + warp < picked ? picks[p0 + warp] : -1;
    using P = Part<ET, VB>;
    int w = 0, first = 0;
    float x[kEach];
    unsigned pass = 0;
    const auto place = [&](int j) { return first + (j / P::kElems * kWarp + lane) * P::kElems + j % P::kElems; };  // of element j
    if (u >= 0) {
      w = u / C;
      first = (u - w * C) * kUnit;
      const char* row = static_cast<const char*>(a.logits) + (row0 + w) * a.row_stride * Elem<ET>::kBytes;
      if (first + kUnit <= a.vocab) {
        P part;
        part.load(row, first, lane);
#pragma unroll
        for (int j = 0; j < kEach; ++j) x[j] = Lanes<VB, ET>::get(part.v[j / P::kElems], j % P::kElems);
      } else {
        using E1 = typename Vec<Elem<ET>::kBytes>::T;
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          x[j] = place(j) < a.vocab ? Lanes<Elem<ET>::kBytes, ET>::get(ld_stream(reinterpret_cast<const E1*>(row) + place(j)), 0) : -INFINITY;
      }
      const float limit = least(w);
#pragma unroll
      for (int j = 0; j < kEach; ++j) pass |= (x[j] >= limit ? 1u : 0u) << j;
      const int more = __reduce_add_sync(0xffffffffu, __popc(pass));
      if (lane == 0 && more > 0) atomicAdd(&s_more, more);
    }
    const auto add = [&](int j) {
      const int at = atomicAdd(&s_count, 1);
      s_x[at] = x[j];
      s_at[at] = (uint32_t)(w * a.vocab + place(j));
    };
    __syncthreads();
    const bool room = s_count + s_more <= kList;
    __syncthreads();
    if (threadIdx.x == 0) s_more = 0;  // the next round adds to it behind the barrier below
    if (room) {
      if (__any_sync(0xffffffffu, pass != 0)) {
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          if (pass >> j & 1) add(j);
      }
      __syncthreads();
      continue;
    }
    // An element of each lane of half of the warps at a time, the list cut to the best n in between.
    for (int j2 = 0; j2 < 2 * kEach; ++j2) {
      __syncthreads();
      const int have = s_count;
      __syncthreads();
      if (have > kList - kJoinThreads / 2) {
        keys_to(have);
        sort_list(s_keys, s_at, have);
        if (have >= n) {
          const Pair last = value_of(s_keys[n - 1]);
          bound = fmaxf(bound, __fadd_rd(last.hi, last.lo));
        }
        done = min(have, n);
        if (threadIdx.x == 0) s_count = done;
        __syncthreads();
      }
      const float limit = least(w);
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (j == j2 / 2 && (warp & 1) == (j2 & 1) && (pass >> j & 1) && x[j] >= limit) add(j);
    }
    __syncthreads();
  }
  const int count = s_count;
  keys_to(count);
  const auto put = [&](int i, int to) {
    const int64_t o = (int64_t)blockIdx.x * n + to;
    const uint32_t V = (uint32_t)a.vocab, w = i >= 0 ? s_at[i] / V : 0;
    a.out_scores[o] = i >= 0 ? value_of(s_keys[i]).hi : -INFINITY;
    a.out_parents[o] = i >= 0 ? (int32_t)(row0 + w) : -1;
    a.out_tokens[o] = i >= 0 ? (int32_t)(s_at[i] - w * V) : -1;
  };
  if (count <= kBests) {  // an entry's place is the number of better ones; four threads count for one
    const int entry = threadIdx.x / 4;
    if (entry - (lane >> 2) < count) {  // the warp has one
      int place = 0;
      const uint64_t own = s_keys[entry];
      const uint32_t at = s_at[entry];
      for (int i = threadIdx.x & 3; i < count; i += 4) place += better(s_keys[i], s_at[i], own, at);
      place += __shfl_xor_sync(0xffffffffu, place, 1);
      place += __shfl_xor_sync(0xffffffffu, place, 2);
      if ((threadIdx.x & 3) == 0 && entry < count && place < n) put(entry, place);
    }
  } else {
    sort_list(s_keys, s_at, count);
    if (threadIdx.x < n) put(threadIdx.x, threadIdx.x);
  }
  if (threadIdx.x < n && (int)threadIdx.x >= count) put(-1, threadIdx.x);
}

template <typename ET, int VB> int launch_select(const SelectArgs& a, cudaStream_t s) {
  const int64_t units = a.requests * a.beams * a.per_row;
  auto k = select_units_kernel<ET, VB>;
  const int64_t work = (units + kThreads / kWarp - 1) / (kThreads / kWarp), most = (int64_t)num_sms() * kUnitCtas;
  launch(k, dim3((unsigned)(work < most ? work : most)), dim3(kThreads), 0, s, a);
  const int rc = check_launch();
  if (rc != MOE_OK) return rc;
  static std::atomic<bool> raised[kSmemDevices];
  auto join = select_join_kernel<ET, VB>;
  if (!allow_smem(join, raised)) return MOE_ERR_CUDA;
  const size_t all = (size_t)a.beams * a.per_row;
  launch(join, dim3((unsigned)a.requests), dim3(kJoinThreads), (all + 1) / 2 * 8 + (all <= kCached ? 8 * all : 0), s, a);
  return check_launch();
}
template <typename ET> int run_select(const SelectArgs& a, cudaStream_t s) {
  const void* ptrs[1] = {a.logits};
  const int64_t stride = a.requests * a.beams > 1 ? a.row_stride * Elem<ET>::kBytes : 0;
  const int vb = pick_vec_bytes(stride, ptrs, 1, Elem<ET>::kBytes);
  if (vb == 16) return launch_select<ET, 16>(a, s);
  if (vb == 8) return launch_select<ET, 8>(a, s);
  if (Elem<ET>::kBytes == 4 || vb == 4) return launch_select<ET, 4>(a, s);
  if constexpr (Elem<ET>::kBytes == 2) return launch_select<ET, 2>(a, s);
  return MOE_ERR_UNSUPPORTED;
}

bool select_ok(int64_t num_requests, int32_t num_beams, int64_t vocab) { return num_requests >= 0 && num_beams >= 1 && vocab >= 1; }
bool select_supported(int64_t num_requests, int32_t num_beams, int64_t vocab) {
  // The last: the second kernel keeps a list of units in shared memory.
  return num_beams <= MOE_BEAM_MAX_BEAMS && vocab <= INT32_MAX && num_beams * vocab <= INT32_MAX &&
         num_requests <= INT32_MAX / num_beams && num_beams * ((vocab + kUnit - 1) / kUnit) <= MOE_BEAM_MAX_UNITS;
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
  if (num_requests > 0 && (num_requests > 1 || num_beams > 1) && row_stride < vocab) return MOE_ERR_INVALID_ARG;
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
