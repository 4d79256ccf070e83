// A mixture-of-experts layer for a few tokens: router, gating, gated experts
// and the weighted sum of their outputs.
//   logits = x router^T; (top_expert, weights) by moe_topk_gating
//   h_a    = weights[a] * silu(g) * u, (g, u) = W_gate_up[e_a] x_t
//   y[t]   = sum_a W_down[e_a] h_a
//
// Every product has few columns (an expert's tokens) and streams its weights
// once, so the layer is bound by the bytes of the experts that the tokens
// reach. Two kernels do the experts: the first writes h (n * F values), the
// second the sum over a token's experts, so that no atomics are needed and
// the order of every sum is fixed. Each CTA sorts the (at most 2048) choices
// by expert itself, in shared memory: that costs about a microsecond and
// spares a launch.
#include <cuda.h>  // types of the tensor maps
#include <math.h>

#include <atomic>
#include <type_traits>

#include "block_common.h"
#include "bulk.cuh"
#include "common.cuh"
#include "moe_block.h"
#include "vec_math.cuh"

namespace moe {
namespace {

struct LayerArgs {
  const void* x;
  const void* w_gate_up;
  const void* w_down;
  const int32_t* top_expert;  // [n]
  const float* weights;       // [n]
  float* h;                   // [n, F], rows in sorted order
  void* y;
  int64_t x_stride, H, F;
  int32_t T, E, K, n;
  int32_t* status;
};

// Lets the next kernel on the stream start while this one runs; it waits for
// this one's end before it reads what this one writes. Called after
// await_previous_kernel() alone (the rules are there); down_stream_kernel calls
// it ahead of its own wait, since the kernel before it has waited.
__device__ __forceinline__ void allow_next_kernel() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------- choices by expert

constexpr int kExpertBits = 16;
static_assert(MOE_GATING_MAX_EXPERTS < 1 << kExpertBits && MOE_LAYER_MAX_CHOICES < 1 << (31 - kExpertBits), "expert and rank in one word");

// The choices sorted by expert (stable), in dynamic shared memory:
// order[i] and token[i]: assignment at sorted place i and its token; the
// active experts, and where each begins in order.
struct Segments {
  int32_t* order;   // [n]
  int32_t* token;   // [n]
  int32_t* expert;  // [min(n, E)]
  int32_t* begin;   // [min(n, E) + 1]
  int32_t active;
};

__host__ __device__ inline size_t segments_bytes(int32_t n, int32_t E) {
  const int m = n < E ? n : E;
  return sizeof(int32_t) * ((size_t)3 * n + E + 2 * m + 2);
}

// Called by the whole CTA: all load the choices and place them, warp 0 ranks them.
__device__ __forceinline__ Segments sort_choices(const int32_t* __restrict__ top_expert, int32_t n, int32_t E, int32_t K,
                                                 int32_t* status, int32_t* smem) {
  const int m = n < E ? n : E;
  Segments s;
  s.order = smem;
  s.token = smem + n;
  int32_t* local = s.token + n;  // a choice's expert, then its rank there above it
  int32_t* count = local + n;  // [E]: choices of the expert, then where they begin
  s.expert = count + E;
  s.begin = s.expert + m;
  int32_t* active = s.begin + m + 1;
  const int lane = lane_id();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    int e = __ldcg(top_expert + i);
    if (e < -1 || e >= E) {
      if (blockIdx.x == 0) flag_status(status, MOE_STATUS_BAD_EXPERT);
      e = -1;
    }
    local[i] = e;
  }
  for (int e = threadIdx.x; e < E; e += blockDim.x) count[e] = 0;
  __syncthreads();
  if (threadIdx.x < kWarp) {
    for (int i0 = 0; i0 < n; i0 += kWarp) {
      const int i = i0 + lane;
      const int e = i < n ? local[i] : -1;
      const unsigned peers = __match_any_sync(0xffffffffu, e);
      if (e >= 0) local[i] = e | (count[e] + __popc(peers & lanemask_lt())) << kExpertBits;
      __syncwarp();
      if (e >= 0 && (peers & lanemask_lt()) == 0) count[e] += __popc(peers);
      __syncwarp();
    }
    int place = 0, found = 0;
    for (int e0 = 0; e0 < E; e0 += kWarp) {
      const int e = e0 + lane;
      const int c = e < E ? count[e] : 0;
      int incl = c;
#pragma unroll
      for (int d = 1; d < kWarp; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, c > 0);
      if (c > 0) {
        const int q = found + __popc(hit & lanemask_lt());
        s.expert[q] = e;
        s.begin[q] = place + incl - c;
      }
      if (e < E) count[e] = place + incl - c;
      place += __shfl_sync(0xffffffffu, incl, kWarp - 1);
      found += __popc(hit);
    }
    if (lane == 0) {
      s.begin[found] = place;
      *active = found;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int v = local[i];
    if (v < 0) continue;
    const int at = count[v & ((1 << kExpertBits) - 1)] + (v >> kExpertBits);
    s.order[at] = i;
    s.token[at] = i / K;
  }
  __syncthreads();
  s.active = *active;
  return s;
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = kWarp / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// ------------------------------------------------- any type, any alignment
//
// Products on the ordinary cores, in fp32, for fp32 layers, small ones and
// rows of fewer than 64 elements: a warp takes four weight rows by four
// tokens, its lanes 16 bytes of each, so that 8 loads feed 16 dot products
// (packed in pairs). Weight rows may begin anywhere (SHIFT): a lane then takes
// the aligned 16-byte piece that holds the first of its elements and shifts it
// together with the next lane's; the last lane's serves its neighbour alone,
// and a row's last piece is masked. These rows, and fp32 ones, come through
// rings of asynchronous copies, four iterations ahead, since two CTAs an SM
// have too few registers for as many loads (fp32, 1501 x 2003, 4 of 16
// experts, 4 and 16 tokens: 131 and 251 us with loads one iteration ahead, 105
// and 214 so, 110 and 222 six ahead; aligned 1504 x 2000, 4 tokens: 109 and
// 101, but 16 tokens of 2048 x 1024, 2 of 8: 72 and 78). Aligned bf16 rows are
// loaded directly: small layers have few iterations (one token 1024 x 2048:
// 15.8 us, with rings 16.9). Loading unaligned rows element by element reached
// a quarter of the rate (5 tokens fp32, 1001 x 777: 26 and 68 us for the two
// kernels). The tokens' rows are aligned, x in the workspace where it is not.

// 16 bytes from global to shared memory, not through L1; zeros when !in (src is not read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / kWarp;
constexpr int kRows = 4;
constexpr int kCols = 4;
template <int N> using Cols = std::integral_constant<int, N>;
constexpr int kSliceChoices = 256;  // up to so many choices, an expert's F may be sliced (its parts lie in shared memory)

__device__ __forceinline__ float f2_sum(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}

// A row of `len` elements read in 16-byte pieces from its first element on.
template <typename ET, bool SHIFT> struct WeightRow {
  static constexpr int kE = 16 / Elem<ET>::kBytes;
  const uint4* p;
  int shift, last, len;  // bytes before the first element in *p; the last piece with an element
  __device__ __forceinline__ WeightRow() {}
  __device__ __forceinline__ WeightRow(const ET* row, int64_t n) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row);
    shift = SHIFT ? (int)(at & 15) : 0;
    p = reinterpret_cast<const uint4*>(at - shift);
    len = (int)n;
    last = (int)((shift + n * Elem<ET>::kBytes - 1) / 16);
  }
  // The aligned piece i to shared memory, where the row has it.
  __device__ __forceinline__ void fetch(uint32_t dst, int i) const {
    if (i <= last) copy16(dst, p + i, true);
  }
  // The elements of piece i from it and the one after it, zeros past the row's end.
  __device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int i) const {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (shift & 8) {
#pragma unroll
      for (int q = 0; q < 6; ++q) w[q] = w[q + 2];
    }
    if (shift & 4) {
#pragma unroll
      for (int q = 0; q < 5; ++q) w[q] = w[q + 1];
    }
    uint4 v;
    v.x = __funnelshift_r(w[0], w[1], 8 * (shift & 3));
    v.y = __funnelshift_r(w[1], w[2], 8 * (shift & 3));
    v.z = __funnelshift_r(w[2], w[3], 8 * (shift & 3));
    v.w = __funnelshift_r(w[3], w[4], 8 * (shift & 3));
    const int left = len - i * kE;  // elements of the row from this piece on
    if (left < kE) {
      v.x &= word_mask(left, 0);
      v.y &= word_mask(left, 1);
      v.z &= word_mask(left, 2);
      v.w &= word_mask(left, 3);
    }
    return v;
  }
  __device__ __forceinline__ static uint32_t word_mask(int left, int word) {
    if constexpr (Elem<ET>::kBytes == 4) return left > word ? 0xffffffffu : 0u;
    const int m = left - 2 * word;
    return m >= 2 ? 0xffffffffu : (m == 1 ? 0xffffu : 0u);
  }
};

// kE elements of a token's row as fp32 pairs: of ET, or fp32 already.
template <typename ET, typename XT> struct TokenRow {
  static constexpr int kE = 16 / Elem<ET>::kBytes;
  static constexpr int kBytes = kE * Elem<XT>::kBytes;
  const char* p;
  __device__ __forceinline__ void get(int i, uint64_t (&out)[kE / 2]) const {
    using V = typename Vec<kBytes>::T;
    const V v = ld_l1(reinterpret_cast<const V*>(p) + i);
#pragma unroll
    for (int q = 0; q < kE / 2; ++q) out[q] = f2_elems<XT>(v, q);
  }
};

// A warp's ring in shared memory: kDepth iterations of kRows pieces a lane.
constexpr int kDepth = 4;
constexpr int kWarpRing = kDepth * kRows * kWarp * 16;
template <typename ET, bool SHIFT> constexpr bool kRing = SHIFT || Elem<ET>::kBytes == 4;
template <typename ET, bool SHIFT> constexpr int kRowsRing = kRing<ET, SHIFT> ? kWarps * kWarpRing : 0;

// Dot products of kRows weight rows with C tokens over pieces [from, to): this
// lane's part. With SHIFT the last lane's piece serves its neighbour alone.
template <int C, typename ET, typename XT, bool SHIFT>
__device__ __forceinline__ void dots(const WeightRow<ET, SHIFT> (&w)[kRows], const TokenRow<ET, XT> (&x)[C], int from, int to,
                                     uint32_t rings, float (&out)[kRows][C]) {
  constexpr int kP = WeightRow<ET, SHIFT>::kE / 2, kStep = SHIFT ? kWarp - 1 : kWarp;
  const int lane = lane_id();
  const uint32_t ring = rings + threadIdx.x / kWarp * kWarpRing + lane * 16;
  uint64_t acc[kRows][C];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
#pragma unroll
    for (int c = 0; c < C; ++c) acc[r][c] = 0ull;
  }
  auto add = [&](const uint4 (&wv)[kRows], const uint64_t (&xv)[C][kP]) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        const uint64_t e = f2_elems<ET>(wv[r], q);
#pragma unroll
        for (int c = 0; c < C; ++c) acc[r][c] = f2_fma(e, xv[c][q], acc[r][c]);
      }
    }
  };
  if constexpr (!kRing<ET, SHIFT>) {
#pragma unroll(C == 1 ? 4 : 2)
    for (int i = from + lane; i < to; i += kWarp) {
      uint4 wv[kRows];
      uint64_t xv[C][kP];
#pragma unroll
      for (int r = 0; r < kRows; ++r) wv[r] = __ldg(w[r].p + i);
#pragma unroll
      for (int c = 0; c < C; ++c) x[c].get(i, xv[c]);
      add(wv, xv);
    }
  } else {
    auto fetch = [&](int slot, int i0) {
      if (i0 < to) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) w[r].fetch(ring + (slot * kRows + r) * (kWarp * 16), i0 + lane);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) fetch(d, from + d * kStep);
    int slot = 0;
    for (int i0 = from; i0 < to; i0 += kStep) {
      const int i = i0 + lane;
      const bool mine = lane < kStep && i < to;
      uint64_t xv[C][kP];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        x[c].get(mine ? i : from, xv[c]);
#pragma unroll
        for (int q = 0; q < kP; ++q) xv[c][q] = mine ? xv[c][q] : 0ull;
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      __syncwarp();
      uint4 wv[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const uint32_t at = ring + (slot * kRows + r) * (kWarp * 16);
        wv[r] = make_uint4(0, 0, 0, 0);
        if (mine) wv[r] = SHIFT ? w[r].shifted(ld_shared16(at), ld_shared16(at + 16), i) : ld_shared16(at);
      }
      __syncwarp();
      fetch(slot, i0 + kDepth * kStep);
      slot = slot + 1 == kDepth ? 0 : slot + 1;
      add(wv, xv);
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
#pragma unroll
    for (int c = 0; c < C; ++c) out[r][c] = f2_sum(acc[r][c]);
  }
}

// x's rows at 16-byte boundaries, padded with zeros to pieces of 16 bytes.
template <typename ET>
__global__ void __launch_bounds__(kThreads) align_rows_kernel(const ET* __restrict__ x, int64_t x_stride, int64_t H, int64_t padded,
                                                              ET* __restrict__ out) {
  await_previous_kernel();
  allow_next_kernel();
  const int64_t t = blockIdx.y;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < padded; i += (int64_t)gridDim.x * kThreads)
    out[t * padded + i] = i < H ? x[t * x_stride + i] : ET(0.0f);
}

// Router logits: a CTA takes kRows experts by kCols tokens, its warps slices of H.
template <typename ET, bool SHIFT>
__global__ void __launch_bounds__(kThreads)
    router_rows_kernel(const ET* __restrict__ x, int64_t x_ld, const ET* __restrict__ router, int64_t H, int32_t T, int32_t E,
                       float* __restrict__ logits) {
  extern __shared__ __align__(16) int32_t smem[];
  __shared__ float part[kWarps][kRows * kCols];
  await_previous_kernel();
  allow_next_kernel();  // the gating, whose few CTAs then wait in place
  const int lane = lane_id(), warp = threadIdx.x / kWarp;
  const int e0 = (int)blockIdx.x * kRows, t0 = (int)blockIdx.y * kCols;
  WeightRow<ET, SHIFT> w[kRows];
  TokenRow<ET, ET> xr[kCols];
#pragma unroll
  for (int r = 0; r < kRows; ++r)  // past the end: the last expert or token again
    w[r] = WeightRow<ET, SHIFT>(router + (int64_t)(e0 + r < E ? e0 + r : E - 1) * H, H);
#pragma unroll
  for (int c = 0; c < kCols; ++c) xr[c].p = reinterpret_cast<const char*>(x + (t0 + c < T ? t0 + c : T - 1) * x_ld);
  const int pieces = (int)((H + w[0].kE - 1) / w[0].kE);
  const int per = ((pieces + kWarps - 1) / kWarps + kWarp - 1) / kWarp * kWarp;
  float acc[kRows][kCols];
  dots(w, xr, warp * per, (warp + 1) * per < pieces ? (warp + 1) * per : pieces, smem_u32(smem), acc);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      const float s = warp_sum(acc[r][c]);
      if (lane == 0) part[warp][r * kCols + c] = s;
    }
  }
  __syncthreads();
  if (threadIdx.x < kRows * kCols) {
    const int r = threadIdx.x / kCols, c = threadIdx.x % kCols;
    float s = 0.0f;
#pragma unroll
    for (int w2 = 0; w2 < kWarps; ++w2) s += part[w2][threadIdx.x];
    if (e0 + r < E && t0 + c < T) logits[(int64_t)(t0 + c) * E + e0 + r] = s;
  }
}

// A warp takes the gate and up rows of two f's of one expert, for all its tokens.
template <typename ET, bool SHIFT>
__global__ void __launch_bounds__(kThreads, 2) gate_up_rows_kernel(LayerArgs a, const ET* __restrict__ x, int64_t x_ld, int64_t h_ld) {
  extern __shared__ __align__(16) int32_t smem[];
  int32_t* const seg = smem + kRowsRing<ET, SHIFT> / sizeof(int32_t);
  await_previous_kernel();
  const Segments s = sort_choices(a.top_expert, a.n, a.E, a.K, a.status, seg);
  const int lane = lane_id();
  const int64_t couples = (a.F + 1) / 2;
  const int pieces = (int)((a.H + WeightRow<ET, SHIFT>::kE - 1) / WeightRow<ET, SHIFT>::kE);
  for (int64_t v = (int64_t)blockIdx.x * kWarps + threadIdx.x / kWarp; v < s.active * couples;
       v += (int64_t)gridDim.x * kWarps) {
    const int q = (int)(v / couples);
    const int64_t f0 = v % couples * 2, f1 = f0 + 1 < a.F ? f0 + 1 : f0;
    const ET* gate = static_cast<const ET*>(a.w_gate_up) + (int64_t)s.expert[q] * 2 * a.F * a.H;
    const ET* up = gate + a.F * a.H;
    const WeightRow<ET, SHIFT> w[kRows] = {{gate + f0 * a.H, a.H}, {gate + f1 * a.H, a.H}, {up + f0 * a.H, a.H}, {up + f1 * a.H, a.H}};
    const int last = s.begin[q + 1] - 1;
    // C tokens from place i0 on; past the last, the last again.
    auto tile = [&](auto cols, int i0) {
      constexpr int C = decltype(cols)::value;
      TokenRow<ET, ET> xr[C];
#pragma unroll
      for (int c = 0; c < C; ++c) xr[c].p = reinterpret_cast<const char*>(x + s.token[i0 + c < last ? i0 + c : last] * x_ld);
      float acc[kRows][C];
      dots(w, xr, 0, pieces, smem_u32(smem), acc);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
#pragma unroll
        for (int c = 0; c < C; ++c) acc[r][c] = warp_sum(acc[r][c]);
      }
      // Lane 2c + f finishes token c's f.
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          if (lane == 2 * c + f && i0 + c <= last && f0 + f < a.F)
            a.h[(i0 + c) * h_ld + f0 + f] = __ldcg(a.weights + s.order[i0 + c]) * (silu(acc[f][c]) * acc[2 + f][c]);
        }
      }
    };
    for (int i0 = s.begin[q]; i0 <= last; i0 += kCols) {
      if (i0 == last)
        tile(Cols<1>(), i0);
      else
        tile(Cols<kCols>(), i0);
    }
    // The places that pad a row of h.
    if (f0 + 2 >= a.F)
      for (int i = s.begin[q]; i <= last; ++i)
        for (int64_t f = a.F + lane; f < h_ld; f += kWarp) a.h[i * h_ld + f] = 0.0f;
  }
}

// A CTA takes kRows columns of y, its warps the active experts (and slices of
// F where those are fewer than the warps); then each token's parts are added
// in the order of its slots.
template <typename ET, bool SHIFT>
__global__ void __launch_bounds__(kThreads, 2) down_rows_kernel(LayerArgs a, int64_t h_ld) {
  extern __shared__ __align__(16) int32_t smem[];
  int32_t* const seg = smem + kRowsRing<ET, SHIFT> / sizeof(int32_t);
  await_previous_kernel();
  const Segments s = sort_choices(a.top_expert, a.n, a.E, a.K, nullptr, seg);
  const int lane = lane_id(), warp = threadIdx.x / kWarp;
  int32_t* place = seg + segments_bytes(a.n, a.E) / sizeof(int32_t);  // [n]: of an assignment, -1 without
  float* part = reinterpret_cast<float*>(place + a.n);                 // [slices][n][kRows]
  for (int i = threadIdx.x; i < a.n; i += kThreads) place[i] = -1;
  __syncthreads();
  const int placed = s.begin[s.active];
  for (int i = threadIdx.x; i < placed; i += kThreads) place[s.order[i]] = i;
  const int slices = a.n <= kSliceChoices && s.active > 0 && s.active < kWarps ? kWarps / s.active : 1;
  const int pieces = (int)((a.F + WeightRow<ET, SHIFT>::kE - 1) / WeightRow<ET, SHIFT>::kE);
  const int per = ((pieces + slices - 1) / slices + kWarp - 1) / kWarp * kWarp;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.H; r0 += (int64_t)gridDim.x * kRows) {
    for (int v = warp; v < s.active * slices; v += kWarps) {
      const int q = v / slices, slice = v % slices;
      const ET* base = static_cast<const ET*>(a.w_down) + (int64_t)s.expert[q] * a.H * a.F;
      WeightRow<ET, SHIFT> w[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) w[r] = WeightRow<ET, SHIFT>(base + (r0 + r < a.H ? r0 + r : a.H - 1) * a.F, a.F);
      const int last = s.begin[q + 1] - 1;
      auto tile = [&](auto cols, int i0) {
        constexpr int C = decltype(cols)::value;
        TokenRow<ET, float> hr[C];
#pragma unroll
        for (int c = 0; c < C; ++c) hr[c].p = reinterpret_cast<const char*>(a.h + (i0 + c < last ? i0 + c : last) * h_ld);
        float acc[kRows][C];
        dots(w, hr, slice * per, (slice + 1) * per < pieces ? (slice + 1) * per : pieces, smem_u32(smem), acc);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const float v2 = warp_sum(acc[r][c]);
            if (lane == r * C + c && i0 + c <= last) part[((int64_t)slice * a.n + i0 + c) * kRows + r] = v2;
          }
        }
      };
      for (int i0 = s.begin[q]; i0 <= last; i0 += kCols) {
        if (i0 == last)
          tile(Cols<1>(), i0);
        else
          tile(Cols<kCols>(), i0);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * kRows; i += kThreads) {
      const int t = i / kRows, r = i % kRows;
      if (r0 + r >= a.H) continue;
      float sum = 0.0f;
      for (int k = 0; k < a.K; ++k) {
        const int at = place[t * a.K + k];
        if (at < 0) continue;
        for (int slice = 0; slice < slices; ++slice) sum += part[((int64_t)slice * a.n + at) * kRows + r];
      }
      if constexpr (Elem<ET>::kBytes == 4)
        static_cast<float*>(a.y)[t * a.H + r0 + r] = sum;
      else
        static_cast<__nv_bfloat16*>(a.y)[t * a.H + r0 + r] = __float2bfloat16_rn(sum);
    }
    __syncthreads();
  }
}

// ---------------------------------------------- bf16 on the tensor cores
//
// Weights stream through a ring of shared-memory stages into the tensor cores:
// tcgen05.mma with 128 weight rows as one operand and an expert's tokens (up
// to 128 at a time) as the other, sums in tensor memory. With few tokens the
// time is that of the weight bytes, so what matters is that copies are always
// in flight: the copying warps run ahead across tiles, rows and experts, and
// the work is cut so that each of the SMs streams the same number of bytes (an
// equal share of the active experts' F gate/up row pairs; about 128 of y's H
// columns for an equal share of the active experts' F), whatever the sizes.
//
// The weights come by tensor copies (TMA) of 4 KB and more, one thread's work.
// The same ring filled with bulk copies of 1 KB pieces of rows reached 4.5
// TB/s (an SM starts one in 34 ns whatever its size), with 16-byte
// asynchronous copies of four warps 5 TB/s (their instructions), with tensor
// copies of 64 elements by 32 rows 7.0 TB/s. The tokens' rows, which lie
// apart, come by 16-byte copies of four warps. Multiplying with
// mma.sync instead of tcgen05 took 1618 us for the first kernel at 128 tokens
// of the Mixtral-8x7B shape (it is bound by its instructions from about 16
// tokens an expert on).
//
// A stage holds one or a few blocks of 64 elements of each row: the weights,
// 128 bytes a row, then the tokens, both in the 128-byte swizzle that the
// tensor copies write and tcgen05 reads (16-byte piece q of row r lies at
// place q ^ (r & 7); blocks start on 1 KB boundaries).
//
// All token warps take part in every stage, each with its rows. Warps that took
// every fourth stage alone would wait for every fourth phase only, and a wait
// tells the phases of a barrier apart by their parity: in a ring of three stages
// such a warp took the phase before last for its own, wrote over a stage in use
// and arrived twice. That ended in a GPU fault.
//
// The sums in tensor memory are fp32, but the tensor cores cut what they add
// where an fp32 addition rounds: over the hundreds of steps of a row, sums come
// out smaller by some 1e-5 of their size (48 tokens, 6144 x 16384: y by 1.9e-5
// on average). Some 1 % of y's bf16 elements are the neighbour of the ones that
// exact sums round to; the error against exact sums is that of the rounding, to
// three digits.
//
// Rows that are not a multiple of 16 bytes, or do not begin on one, are out of
// reach of tensor copies: 16 warps copy and shift their pieces.
//
// Warps: 0..3 take sums out of tensor memory (warp w its lanes 32w ..), 4..7
// copy tokens, 8 (SHIFT: 8..23) copies weights, the last issues the products.
// Sums are double buffered. Every wait is bounded: a warp that gives up sets
// MOE_STATUS_TIMEOUT and does no more work, nor lets others go on (it arrives
// nowhere), so that they give up in turn. The warps that take sums out write
// NaN where theirs did not come: to h, whence it reaches the rows of y of that
// expert's tokens, or to the sums of y. All warps meet at the end, where copies
// and products still in flight are waited for (bounded again) and the tensor
// memory is freed.

constexpr int kOutWarps = 4;
constexpr int kTokenWarps = 4;
constexpr int kCopyWarp = kOutWarps + kTokenWarps;  // the first
template <bool SHIFT> constexpr int kCopyWarps = SHIFT ? 16 : 1;
template <bool SHIFT> constexpr int kMulWarp = kCopyWarp + kCopyWarps<SHIFT>;
template <bool SHIFT> constexpr int kStreamThreads = (kMulWarp<SHIFT> + 1) * kWarp;
constexpr int kMaxStages = 8;
constexpr int kBlock = 64;       // elements of a block: the 128 bytes of a swizzled row
constexpr int kRowBytes = 128;
constexpr int kTileRows = 128;   // weight rows of a product
constexpr int kMaxTokens = 128;  // of an expert at a time (256 tokens of the Mixtral-8x7B shape: 788 us, with 64: 985)
constexpr uint64_t kWaitNs = 2000000000;  // after which a wait gives up
constexpr uint64_t kTestWaitNs = 20000000;  // the same while moe_test_block_waits makes some give up at once

__device__ __forceinline__ uint32_t align_1k(uint32_t p) { return (p + 1023u) & ~1023u; }
__host__ __device__ constexpr int round_to(int v, int m) { return (v + m - 1) / m * m; }

__device__ __forceinline__ void mbar_init_count(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A box of the tensor from coordinates (x, y, z); x is a multiple of 64.
__device__ __forceinline__ void tensor_copy(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2,%3,%4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t dst, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// The thread's arrival on the barrier, once all its copies so far have landed.
__device__ __forceinline__ void arrive_after_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// True in one lane of a converged warp. Tensor copies and products are issued
// behind this and not behind a test of the lane's number: the compiler then
// knows that one lane issues them (237 against 104 clocks a product, 44 with
// the four of a block unrolled).
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// Tensor memory: allocation by one warp, whose address lands in shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Eight columns from `at` on: lane l of the warp gets its row's.
__device__ __forceinline__ void tmem_load8(float (&v)[8], uint32_t at) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// Arrives on the barrier when this thread's products so far are done.
__device__ __forceinline__ void products_arrive(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// Descriptor of a block in shared memory: rows of 128 bytes along k, 128-byte
// swizzle, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t block_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// sums[128 rows][n columns] (+)= 16 elements of each row by 16 of each column; bf16, fp32 sums.
__device__ __forceinline__ void product(uint32_t sums, uint64_t rows, uint64_t cols, int n, bool add) {
  const uint32_t kind = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((kTileRows >> 4) << 24);
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(sums),
      "l"(rows), "l"(cols), "r"(kind), "r"((uint32_t)add)
      : "memory");
}

// Where a warp stands in the ring of stages or in the two buffers of sums, and
// how many it has done.
struct Ring {
  int n, i;
  uint32_t parity;
  int done;
  __device__ __forceinline__ Ring(int n_, uint32_t parity_) : n(n_), i(0), parity(parity_), done(0) {}
  __device__ __forceinline__ void advance() {
    ++done;
    if (++i == n) {
      i = 0;
      parity ^= 1;
    }
  }
};

struct StreamArgs {
  LayerArgs a;
  __nv_bfloat16* h_hi;  // [n, h_ld] in sorted order: h = h_hi + h_lo, zeros past F
  __nv_bfloat16* h_lo;
  int64_t h_ld;
  float* parts;  // [slices, T, H]: the slices' sums, where there are more than two
  int64_t parts_ld;
  uint32_t give_up;  // kGiveUp*: 0 but in tests
};
// A kernel's cut of its work and of its shared memory.
struct StreamShape {
  int stages, stage_bytes, blocks;  // blocks of 64 elements in a stage
  int tokens;                       // of an expert at a time (a multiple of 16, the products' columns; 8 in the second kernel)
  int rows;                         // weight rows of a tile (first kernel: two for each gate/up pair)
  int slices;                       // second kernel: CTAs that share a tile's experts and elements
  uint32_t cols;                    // tensor memory columns
};

struct StreamShared {
  uint64_t full[kMaxStages], empty[kMaxStages], sums_full[2], sums_empty[2];
  uint32_t tmem;
  int issued;  // stages whose weights are on their way, set when a warp has given up
};

template <bool SHIFT> __device__ __forceinline__ void init_shared(StreamShared& sh, int stages) {
  for (int i = 0; i < stages; ++i) {
    mbar_init_count(smem_u32(&sh.full[i]), kTokenWarps * kWarp + (SHIFT ? kCopyWarps<true> * kWarp : 1));  // the tokens' copies and the weights'
    mbar_init_count(smem_u32(&sh.empty[i]), 1);
  }
  for (int i = 0; i < 2; ++i) {
    mbar_init_count(smem_u32(&sh.sums_full[i]), 1);
    mbar_init_count(smem_u32(&sh.sums_empty[i]), kOutWarps);
  }
  fence_mbarrier_init();
}

// How long a warp waits.
struct Patience {
  int polls;
  uint64_t ns;
  int32_t* status;
  __device__ __forceinline__ Patience(int32_t* status_) : polls(kSpinLimit), ns(kWaitNs), status(status_) {}
  __device__ __forceinline__ Patience(const StreamArgs& p, uint32_t who)
      : polls(p.give_up & who ? 0 : kSpinLimit), ns(p.give_up ? kTestWaitNs : kWaitNs), status(p.a.status) {}
};

// By a whole warp, bounded in polls and in time; false once a wait has given up.
__device__ __forceinline__ bool wait_bar(bool ok, uint64_t* bar, uint32_t parity, const Patience& patience) {
  if (!ok) return false;
  const uint32_t at = smem_u32(bar);
  uint64_t since = 0;
  ok = false;
  for (int it = 0; it < patience.polls; ++it) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(at), "r"(parity)
        : "memory");
    if (__all_sync(0xffffffffu, done != 0)) {
      ok = true;
      break;
    }
    if ((it & 255) == 255) {
      uint64_t now;
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
      now = __shfl_sync(0xffffffffu, now, 0);
      if (since == 0) since = now;
      if (now - since > patience.ns) break;
    }
  }
  if (!ok && lane_id() == 0) flag_status(patience.status, MOE_STATUS_TIMEOUT);
  return ok;
}

// The products of every stage, one thread's work. WALK: tiles and their
// stages; `columns(w)`: columns of a tile's products; `tokens_at(w)`: offset of
// the tokens in a stage; block: bytes of a block of weight rows.
template <typename WALK, typename C, typename O>
__device__ __forceinline__ bool multiply(WALK w, StreamShared& sh, const StreamShape& z, uint32_t ring, int block,
                                         const Patience& patience, C columns, O tokens_at) {
  Ring r(z.stages, 0), d(2, 1);
  const uint32_t tmem = sh.tmem;
  bool ok = true;
  while (w.more()) {
    ok = wait_bar(ok, &sh.sums_empty[d.i], d.parity, patience);
    tmem_fence_after();
    const int n = columns(w);
    bool add = false;
    for (bool last = false; ok && !last; w.next(), r.advance()) {
      last = w.last_stage();
      ok = wait_bar(ok, &sh.full[r.i], r.parity, patience);
      if (!ok) break;
      fence_async_shared();  // the tokens' copies were ordinary writes; the products read by another path
      tmem_fence_after();
      __syncwarp();
      if (elect_lane()) {
        const uint32_t at = ring + r.i * z.stage_bytes, sums = tmem + d.i * (z.cols / 2);
        const uint32_t tokens = at + tokens_at(w);
        const int kc = w.kc();
        for (int b = 0; b * kBlock < kc; ++b) {
          const uint64_t rows = block_desc(at + b * block), cols = block_desc(tokens + b * n * kRowBytes);
          // 16 elements are 32 bytes: 2 in the descriptor.
          if (kc - b * kBlock >= kBlock) {
#pragma unroll
            for (int k = 0; k < kBlock / 16; ++k) product(sums, rows + 2 * k, cols + 2 * k, n, k > 0 || add);
          } else {
            for (int k = 0; k * 16 < kc - b * kBlock; ++k) product(sums, rows + 2 * k, cols + 2 * k, n, k > 0 || add);
          }
          add = true;
        }
        products_arrive(smem_u32(&sh.empty[r.i]));
        if (last) products_arrive(smem_u32(&sh.sums_full[d.i]));
      }
      add = true;
      __syncwarp();
    }
    if (!ok) break;
    d.advance();
  }
  // Every product is done and every arrival lands before the CTA may end, also
  // after giving up: of the stages' last uses, and of the sums' (whose barriers'
  // phases begin where sums_empty's second ones do).
  const Patience last(patience.status);
  for (int i = 0; i < z.stages; ++i) ok = wait_bar(true, &sh.empty[i], i < r.i ? r.parity : r.parity ^ 1, last) && ok;
  for (int i = 0; i < 2; ++i) ok = wait_bar(true, &sh.sums_full[i], i < d.i ? d.parity ^ 1 : d.parity, last) && ok;
  return ok;
}

// The end of a CTA's work, for all its threads: `ok` false in the warps that
// gave up; r: where the warps that copy stand. A tensor copy in flight would
// write to memory that is another CTA's by then, so its barrier's phase is
// waited for; the token warps first arrive for the stages that they left.
template <bool SHIFT> __device__ __forceinline__ void meet(StreamShared& sh, int warp, bool ok, Ring& r, int32_t* status) {
  tmem_fence_before();
  const bool failed = __syncthreads_or(!ok);
  tmem_fence_after();
  if (SHIFT || !failed) return;
  if (threadIdx.x == kCopyWarp * kWarp) sh.issued = r.done;
  __syncthreads();
  if (warp >= kOutWarps && warp < kCopyWarp)
    for (; r.done < sh.issued; r.advance()) mbar_arrive(smem_u32(&sh.full[r.i]));
  if (warp == kCopyWarp)
    for (int i = 0; i < r.n; ++i) wait_bar(true, &sh.full[i], i < r.i ? r.parity ^ 1 : r.parity, Patience(status));
  __syncthreads();
}

// The weights of every stage where rows are not a multiple of 16 bytes (or do
// not begin on one). A warp copies the aligned 16-byte pieces that hold a
// stage's elements of its rows into a buffer of its own, kRawDepth stages
// ahead; then its lanes shift two neighbouring pieces of a row together and
// store them where tensor copies would. Pieces held in registers instead, one
// stage ahead: 8 tokens, 2045 x 8191, 2 of 16 experts, 386 us; 291 so (three
// stages ahead, in stages of two blocks: no better). The ordinary cores took
// 469 for it, and 2177 instead of 577 for 48 tokens, 4093 x 4099, 4 of 16.
// ROWS: where this warp's i-th row of a tile begins (first(w) + i * step
// bytes), how many it has, and the i-th's place in the tile; len: elements of
// a row.
constexpr int kRawDepth = 2;
constexpr int kEach = kTileRows / kCopyWarps<true>;  // rows of a copying warp
__host__ __device__ constexpr int raw_row(int blocks) { return blocks * kRowBytes + 16; }
__host__ __device__ constexpr int raw_bytes(int blocks) { return kRawDepth * kTileRows * raw_row(blocks); }

template <typename WALK, typename ROWS>
__device__ __forceinline__ bool copy_shifted(WALK w, StreamShared& sh, const StreamShape& z, uint32_t ring, int block, int64_t len,
                                             const Patience& patience, const ROWS& rows) {
  const int lane = lane_id(), row_bytes = raw_row(z.blocks);
  const uint32_t raw = ring + z.stages * z.stage_bytes + (threadIdx.x / kWarp - kCopyWarp) * (kRawDepth * kEach) * row_bytes + lane * 16;
  const bool mine = lane < z.blocks * 8;
  WALK ahead = w;
  auto fetch = [&](int slot) {
    if (ahead.more()) {
      const int n = rows.count(ahead), pieces = (ahead.kc() + 7) / 8, left = (int)(len - ahead.k0) - lane * 8;
      uintptr_t from = rows.first(ahead) + 2 * ahead.k0;
      const uint32_t dst = raw + slot * kEach * row_bytes;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int shift = (int)(from & 15);
        if (i < n && lane <= pieces && 2 * left + shift > 0)
          copy16(dst + i * row_bytes, reinterpret_cast<const void*>(from - shift + 16 * lane), true);
        from += rows.step;
      }
      ahead.next();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int d = 0; d < kRawDepth; ++d) fetch(d);
  bool ok = true;
  int slot = 0;
  for (Ring r(z.stages, 1); w.more(); w.next(), r.advance()) {
    const int n = rows.count(w), left = (int)(len - w.k0) - lane * 8;  // elements of the row from this lane's piece on
    const int shift0 = (int)((rows.first(w) + 2 * w.k0) & 15);
    asm volatile("cp.async.wait_group %0;" ::"n"(kRawDepth - 1) : "memory");
    ok = wait_bar(ok, &sh.empty[r.i], r.parity, patience);
    if (!ok) break;
    __syncwarp();
    const uint32_t stage = ring + r.i * z.stage_bytes + (lane >> 3) * block, src = raw + slot * kEach * row_bytes;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (mine && i < n) {
        const int shift = (shift0 + i * (int)(rows.step & 15)) & 15, bits = 8 * (shift & 3);
        const uint4 v = ld_shared16(src + i * row_bytes), next = ld_shared16(src + i * row_bytes + 16);
        // The shift is the same in all lanes.
        const bool by8 = shift & 8, by4 = shift & 4;
        const uint32_t a0 = by8 ? v.z : v.x, a1 = by8 ? v.w : v.y, a2 = by8 ? next.x : v.z, a3 = by8 ? next.y : v.w,
                       a4 = by8 ? next.z : next.x, a5 = by8 ? next.w : next.y;
        const uint32_t u0 = by4 ? a1 : a0, u1 = by4 ? a2 : a1, u2 = by4 ? a3 : a2, u3 = by4 ? a4 : a3, u4 = by4 ? a5 : a4;
        uint4 o;
        o.x = __funnelshift_r(u0, u1, bits);
        o.y = __funnelshift_r(u1, u2, bits);
        o.z = __funnelshift_r(u2, u3, bits);
        o.w = __funnelshift_r(u3, u4, bits);
        if (left < 8) {  // beyond the row: zeros
          o.x &= WeightRow<__nv_bfloat16, true>::word_mask(left, 0);
          o.y &= WeightRow<__nv_bfloat16, true>::word_mask(left, 1);
          o.z &= WeightRow<__nv_bfloat16, true>::word_mask(left, 2);
          o.w &= WeightRow<__nv_bfloat16, true>::word_mask(left, 3);
        }
        const int at = rows.place(i);
        st_shared16(stage + at * kRowBytes + (((lane ^ at) & 7) << 4), o);
      }
    }
    __syncwarp();
    fetch(slot);
    slot = slot + 1 == kRawDepth ? 0 : slot + 1;
    fence_async_shared();
    mbar_arrive(smem_u32(&sh.full[r.i]));
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  return ok;
}

// Tiles of up to z.rows / 2 row pairs (gate, up) of one expert by up to
// z.tokens of its tokens, over the whole of H. A box has 16 pairs: those beyond a CTA's
// share are read too (their owner reads them as well) and left.
struct GateUpWalk {
  const Segments& s;
  int64_t pos, end, F, f0;
  int q, nf, i0, ntok, K, k0, per_stage, per_pass, pairs;
  __device__ GateUpWalk(const Segments& s_, const LayerArgs& a, const StreamShape& z)
      : s(s_), F(a.F), K((int)a.H), per_stage(z.blocks * kBlock), per_pass(z.tokens), pairs(z.rows / 2) {
    const int64_t rows = s.active * F;
    pos = rows * blockIdx.x / gridDim.x;
    end = rows * (blockIdx.x + 1) / gridDim.x;
    if (pos < end) tile();
  }
  __device__ __forceinline__ bool more() const { return pos < end; }
  __device__ __forceinline__ void tile() {
    q = (int)(pos / F);
    f0 = pos - q * F;
    const int64_t m = end - pos < F - f0 ? end - pos : F - f0;
    nf = m < pairs ? (int)m : pairs;
    i0 = s.begin[q];
    pass();
  }
  __device__ __forceinline__ void pass() {
    const int left = s.begin[q + 1] - i0;
    ntok = left < per_pass ? left : per_pass;
    k0 = 0;
  }
  __device__ __forceinline__ int kc() const { return K - k0 < per_stage ? K - k0 : per_stage; }
  __device__ __forceinline__ bool last_stage() const { return k0 + per_stage >= K; }
  __device__ __forceinline__ void next() {
    k0 += per_stage;
    if (k0 < K) return;
    i0 += ntok;
    if (i0 < s.begin[q + 1]) return pass();
    pos += nf;
    if (pos < end) tile();
  }
  __device__ __forceinline__ void next_pass() {
    k0 = K;
    next();
  }
};

// Rows of a copying warp: even warps gate rows, odd ones up rows, every eighth.
struct GateUpRows {
  const Segments& s;
  uintptr_t base;
  int64_t F, H, step;
  int up, f;
  __device__ GateUpRows(const Segments& s_, const LayerArgs& a, int warp)
      : s(s_), base(reinterpret_cast<uintptr_t>(a.w_gate_up)), F(a.F), H(a.H), step(16 * a.H), up(warp & 1), f(warp >> 1) {}
  __device__ __forceinline__ uintptr_t first(const GateUpWalk& w) const {
    return base + 2 * (((2 * s.expert[w.q] + up) * F + w.f0 + f) * H);
  }
  __device__ __forceinline__ int count(const GateUpWalk& w) const { return (w.nf - f + 7) >> 3; }
  __device__ __forceinline__ int place(int i) const { return (i >> 1) * 32 + (i & 1) * 8 + up * 16 + f; }
};

template <bool SHIFT>
__global__ void __launch_bounds__(kStreamThreads<SHIFT>)
    gate_up_stream_kernel(StreamArgs p, StreamShape z, const __grid_constant__ CUtensorMap map) {
  extern __shared__ __align__(1024) unsigned char dyn[];
  __shared__ StreamShared sh;
  const LayerArgs& a = p.a;
  const int block = z.rows * kRowBytes;
  const int warp = threadIdx.x / kWarp, lane = lane_id();
  if (warp == kMulWarp<SHIFT>) tmem_alloc(smem_u32(&sh.tmem), z.cols);
  if (threadIdx.x == kCopyWarp * kWarp) {
    if constexpr (!SHIFT) prefetch_map(&map);
    init_shared<SHIFT>(sh, z.stages);
  }
  await_previous_kernel();
  const uint32_t ring = align_1k(smem_u32(dyn));
  unsigned char* rest = dyn + (ring - smem_u32(dyn)) + (size_t)z.stages * z.stage_bytes + (SHIFT ? raw_bytes(z.blocks) : 0);
  tmem_fence_before();
  const Segments s = sort_choices(a.top_expert, a.n, a.E, a.K, a.status,
                                  reinterpret_cast<int32_t*>(rest));
  tmem_fence_after();
  allow_next_kernel();
  GateUpWalk w(s, a, z);
  bool ok = true;
  Ring r(z.stages, 1);  // of the warps that copy
  if (SHIFT && warp >= kCopyWarp && warp < kMulWarp<SHIFT>) {
    ok = copy_shifted(w, sh, z, ring, block, a.H, Patience(p, kGiveUpWeights), GateUpRows(s, a, warp - kCopyWarp));
  } else if (!SHIFT && warp == kCopyWarp) {
    for (const Patience patience(p, kGiveUpWeights); w.more(); w.next(), r.advance()) {
      ok = wait_bar(ok, &sh.empty[r.i], r.parity, patience);
      if (!ok) break;
      __syncwarp();
      if (elect_lane()) {
        const uint32_t bar = smem_u32(&sh.full[r.i]), at = ring + r.i * z.stage_bytes;
        const int n = (w.kc() + kBlock - 1) / kBlock, boxes = (w.nf + 15) / 16, e = s.expert[w.q];
        mbar_expect(bar, n * boxes * 32 * kRowBytes);
        for (int b = 0; b < n; ++b)
          for (int g = 0; g < boxes; ++g)
            tensor_copy(at + b * block + g * 32 * kRowBytes, &map, w.k0 + b * kBlock, (int)w.f0 + g * 16, 2 * e, bar);
      }
    }
  } else if (warp == kMulWarp<SHIFT>) {
    ok = multiply(w, sh, z, ring, block, Patience(p, kGiveUpProducts), [](const GateUpWalk& v) { return round_to(v.ntok, 16); },
             [&](const GateUpWalk&) { return z.blocks * block; });
  } else if (warp >= kOutWarps) {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x);
    const int piece = lane & 7, first = (warp - kOutWarps) * 4 + (lane >> 3);
    for (const Patience patience(p, kGiveUpTokens); w.more(); w.next(), r.advance()) {
      ok = wait_bar(ok, &sh.empty[r.i], r.parity, patience);
      if (!ok) break;
      const uint32_t at = ring + r.i * z.stage_bytes + z.blocks * block;
      const int kc = w.kc(), n = round_to(w.ntok, 16);
      for (int i = first; i < w.ntok; i += 4 * kTokenWarps) {
        const __nv_bfloat16* src = x + s.token[w.i0 + i] * a.x_stride + w.k0 + piece * 8;
        const uint32_t dst = at + i * kRowBytes + ((piece ^ (i & 7)) << 4);
        for (int b = 0; b * kBlock < kc; ++b) {
          const bool in = b * kBlock + piece * 8 < kc;
          copy16(dst + b * n * kRowBytes, in ? src + b * kBlock : x, in);
        }
      }
      arrive_after_copies(smem_u32(&sh.full[r.i]));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // Rows of the sums: 16 gate rows, their 16 up rows, the next 16 gate rows ...
    const bool gate = lane < 16;
    const int f = warp * 16 + (lane & 15);
    const Patience patience(p, kGiveUpSums);
    for (Ring d(2, 0); w.more(); w.next_pass(), d.advance()) {
      ok = wait_bar(ok, &sh.sums_full[d.i], d.parity, patience);
      tmem_fence_after();
      if (ok && warp * 16 < w.nf) {
        const uint32_t at = sh.tmem + d.i * (z.cols / 2) + ((uint32_t)(warp * 32) << 16);
        for (int c0 = 0; c0 < w.ntok; c0 += 8) {
          float v[8];
          __syncwarp();
          tmem_load8(v, at + c0);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // Lower lanes finish columns 0..3, upper lanes 4..7.
            const float other = __shfl_xor_sync(0xffffffffu, gate ? v[c + 4] : v[c], 16);
            const float g = gate ? v[c] : other, u = gate ? other : v[c + 4];
            const int col = c0 + c + (gate ? 0 : 4);
            if (f < w.nf && col < w.ntok) {
              const int i = w.i0 + col;
              const float h = __ldcg(a.weights + s.order[i]) * (silu(g) * u);
              // Two bf16 numbers keep 16 significant bits of h: 2^-16 of it is lost at most, where y's own
              // rounding loses 2^-8. One alone would round the layer's result twice; three would make the
              // second kernel's columns half as many again.
              const __nv_bfloat16 hi = __float2bfloat16_rn(h);
              const float rest = h - __bfloat162float(hi);
              p.h_hi[i * p.h_ld + w.f0 + f] = hi;
              p.h_lo[i * p.h_ld + w.f0 + f] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.0f);
            }
          }
        }
      }
      if (!ok && f < w.nf) {
        for (int i = w.i0 + (gate ? 0 : 1); i < w.i0 + w.ntok; i += 2)
          p.h_hi[i * p.h_ld + w.f0 + f] = p.h_lo[i * p.h_ld + w.f0 + f] = __float2bfloat16_rn(__int_as_float(0x7fffffff));
      }
      if (SHIFT && warp == 0 && w.f0 + w.nf == a.F && lane < p.h_ld - a.F) {
        for (int i = w.i0; i < w.i0 + w.ntok; ++i)
          p.h_hi[i * p.h_ld + a.F + lane] = p.h_lo[i * p.h_ld + a.F + lane] = __float2bfloat16_rn(0.0f);
      }
      tmem_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(smem_u32(&sh.sums_empty[d.i]));
    }
  }
  meet<SHIFT>(sh, warp, ok, r, a.status);
  if (warp == kMulWarp<SHIFT>) tmem_free(sh.tmem, z.cols);
}

// y's columns [r0, r0 + nr) for one expert's tokens after another, over this
// slice's range of all experts' blocks (all of them without slices).
struct DownWalk {
  const Segments& s;
  int64_t r0, end;
  int nr, q, i0, ntok, K0, K, k0, per_stage, per_pass, rows, F, blocks, first, last;
  __device__ DownWalk(const Segments& s_, const LayerArgs& a, const StreamShape& z)
      : s(s_), per_stage(z.blocks * kBlock), per_pass(z.tokens), rows(z.rows), F((int)a.F), blocks((F + kBlock - 1) / kBlock) {
    const int64_t tiles = gridDim.x / z.slices, tile_id = blockIdx.x / z.slices, slice = blockIdx.x % z.slices;
    r0 = a.H * tile_id / tiles;
    end = a.H * (tile_id + 1) / tiles;
    first = (int)((int64_t)s.active * blocks * slice / z.slices);
    last = (int)((int64_t)s.active * blocks * (slice + 1) / z.slices);
    if (first >= last) r0 = end;
    if (more()) tile();
  }
  __device__ __forceinline__ bool more() const { return r0 < end; }
  __device__ __forceinline__ void tile() {
    nr = end - r0 < rows ? (int)(end - r0) : rows;
    q = first / blocks;
    expert();
  }
  __device__ __forceinline__ void expert() {
    const int from = q * blocks;
    K0 = (first > from ? first - from : 0) * kBlock;
    K = last - from < blocks ? (last - from) * kBlock : F;
    i0 = s.begin[q];
    pass();
  }
  __device__ __forceinline__ void pass() {
    const int left = s.begin[q + 1] - i0;
    ntok = left < per_pass ? left : per_pass;
    k0 = K0;
  }
  __device__ __forceinline__ int kc() const { return K - k0 < per_stage ? K - k0 : per_stage; }
  __device__ __forceinline__ bool last_stage() const { return k0 + per_stage >= K; }
  __device__ __forceinline__ void next() {
    k0 += per_stage;
    if (k0 < K) return;
    i0 += ntok;
    if (i0 < s.begin[q + 1]) return pass();
    if (++q * blocks < last) return expert();
    r0 += nr;
    if (r0 < end) tile();
  }
  __device__ __forceinline__ void next_pass() {
    k0 = K;
    next();
  }
};

// Rows of a copying warp: every sixteenth.
struct DownRows {
  const Segments& s;
  uintptr_t base;
  int64_t F, H, step;
  int warp;
  __device__ DownRows(const Segments& s_, const LayerArgs& a, int warp_)
      : s(s_), base(reinterpret_cast<uintptr_t>(a.w_down)), F(a.F), H(a.H), step(32 * a.F), warp(warp_) {}
  __device__ __forceinline__ uintptr_t first(const DownWalk& w) const { return base + 2 * ((s.expert[w.q] * H + w.r0 + warp) * F); }
  __device__ __forceinline__ int count(const DownWalk& w) const { return (w.nr - warp + 15) >> 4; }
  __device__ __forceinline__ int place(int i) const { return i * 16 + warp; }
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// A float of another CTA of the cluster, at the place where this CTA has `p`.
__device__ __forceinline__ float load_peer(const float* p, uint32_t rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

template <bool SHIFT>
__global__ void __launch_bounds__(kStreamThreads<SHIFT>)
    down_stream_kernel(StreamArgs p, StreamShape z, const __grid_constant__ CUtensorMap map) {
  extern __shared__ __align__(1024) unsigned char dyn[];
  __shared__ StreamShared sh;
  const LayerArgs& a = p.a;
  const int warp = threadIdx.x / kWarp, lane = lane_id();
  // The gate/up kernel has waited for all before it, so the routing may be
  // read and weights copied while it still runs (a CTA starts as one of the
  // other kernel leaves its SM); h may not be read.
  if (warp == kMulWarp<SHIFT>) tmem_alloc(smem_u32(&sh.tmem), z.cols);
  if (threadIdx.x == kCopyWarp * kWarp) {
    if constexpr (!SHIFT) prefetch_map(&map);
    init_shared<SHIFT>(sh, z.stages);
  }
  const uint32_t ring = align_1k(smem_u32(dyn));
  unsigned char* rest = dyn + (ring - smem_u32(dyn)) + (size_t)z.stages * z.stage_bytes + (SHIFT ? raw_bytes(z.blocks) : 0);
  int32_t* seg = reinterpret_cast<int32_t*>(rest);
  tmem_fence_before();
  const Segments s = sort_choices(a.top_expert, a.n, a.E, a.K, nullptr, seg);
  tmem_fence_after();
  allow_next_kernel();
  // [T, z.rows]: with a stride that is the same for all of a CTA's tiles, each
  // thread meets its own places alone, in every tile, and the warps that add the
  // sums need no barrier between tiles (with a tile's own number of columns for
  // a stride, the next tile's places are other warps' in the one before).
  float* ysum = reinterpret_cast<float*>(seg + segments_bytes(a.n, a.E) / sizeof(int32_t));
  DownWalk w(s, a, z);
  const int block = round_to(z.rows, 8) * kRowBytes;
  bool ok = true;
  Ring r(z.stages, 1);  // of the warps that copy
  if (SHIFT && warp >= kCopyWarp && warp < kMulWarp<SHIFT>) {
    ok = copy_shifted(w, sh, z, ring, block, a.F, Patience(p, kGiveUpWeights), DownRows(s, a, warp - kCopyWarp));
  } else if (!SHIFT && warp == kCopyWarp) {
    for (const Patience patience(p, kGiveUpWeights); w.more(); w.next(), r.advance()) {
      ok = wait_bar(ok, &sh.empty[r.i], r.parity, patience);
      if (!ok) break;
      __syncwarp();
      if (elect_lane()) {
        const uint32_t bar = smem_u32(&sh.full[r.i]), at = ring + r.i * z.stage_bytes;
        const int n = (w.kc() + kBlock - 1) / kBlock;
        mbar_expect(bar, n * z.rows * kRowBytes);
        for (int b = 0; b < n; ++b)
          tensor_copy(at + b * block, &map, w.k0 + b * kBlock, (int)w.r0, s.expert[w.q], bar);
      }
    }
  } else if (warp == kMulWarp<SHIFT>) {
    // The tile reads 128 rows; what lies beyond its weights lands in rows of the sums that nobody reads.
    ok = multiply(w, sh, z, ring, block, Patience(p, kGiveUpProducts), [](const DownWalk& v) { return 2 * round_to(v.ntok, 8); },
             [&](const DownWalk&) { return z.blocks * block; });
  } else if (warp >= kOutWarps) {
    await_previous_kernel();
    const int piece = lane & 7, first = (warp - kOutWarps) * 4 + (lane >> 3);
    for (const Patience patience(p, kGiveUpTokens); w.more(); w.next(), r.advance()) {
      ok = wait_bar(ok, &sh.empty[r.i], r.parity, patience);
      if (!ok) break;
      // Columns: the tokens' high parts, then from a multiple of 8 on their low parts.
      const uint32_t at = ring + r.i * z.stage_bytes + z.blocks * block;
      const int kc = w.kc(), n = round_to(w.ntok, 8);
      for (int i = first; i < w.ntok; i += 4 * kTokenWarps) {
        const int64_t from = (w.i0 + i) * p.h_ld + w.k0 + piece * 8;
        const uint32_t dst = at + i * kRowBytes + ((piece ^ (i & 7)) << 4);
        for (int b = 0; b * kBlock < kc; ++b) {
          const bool in = b * kBlock + piece * 8 < kc;
          copy16(dst + b * 2 * n * kRowBytes, in ? p.h_hi + from + b * kBlock : p.h_hi, in);
          copy16(dst + (b * 2 + 1) * n * kRowBytes, in ? p.h_lo + from + b * kBlock : p.h_lo, in);
        }
      }
      arrive_after_copies(smem_u32(&sh.full[r.i]));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    const int64_t tiles = gridDim.x / z.slices, tile_id = blockIdx.x / z.slices;
    const int64_t r_end = a.H * (tile_id + 1) / tiles;
    const int row = threadIdx.x;  // of the tile: this thread's sums, for every token
    const Patience patience(p, kGiveUpSums);
    Ring d(2, 0);
    for (int64_t r0 = a.H * tile_id / tiles; r0 < r_end; r0 += z.rows) {
      const int nr = r_end - r0 < z.rows ? (int)(r_end - r0) : z.rows;
      if (row < nr)
        for (int t = 0; t < a.T; ++t) ysum[t * z.rows + row] = 0.0f;
      for (; w.more() && w.r0 == r0; w.next_pass(), d.advance()) {
        ok = wait_bar(ok, &sh.sums_full[d.i], d.parity, patience);
        tmem_fence_after();
        if (ok && warp * 32 < nr) {
          const uint32_t at = sh.tmem + d.i * (z.cols / 2) + ((uint32_t)(warp * 32) << 16);
          const int n = round_to(w.ntok, 8);
          for (int c0 = 0; c0 < w.ntok; c0 += 8) {
            float hi[8], lo[8];
            __syncwarp();
            tmem_load8(hi, at + c0);
            tmem_load8(lo, at + n + c0);
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (row < nr && c0 + c < w.ntok) ysum[s.token[w.i0 + c0 + c] * z.rows + row] += hi[c] + lo[c];
          }
        }
        tmem_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(smem_u32(&sh.sums_empty[d.i]));
      }
      if (!ok && row < nr)
        for (int t = 0; t < a.T; ++t) ysum[t * z.rows + row] = __int_as_float(0x7fffffff);
      if (row < nr && z.slices == 1) {
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + r0 + row;
        for (int t = 0; t < a.T; ++t) y[t * a.H] = __float2bfloat16_rn(ysum[t * z.rows + row]);
      } else if (row < nr && z.slices > 2) {
        float* part = p.parts + blockIdx.x % z.slices * p.parts_ld + r0 + row;
        for (int t = 0; t < a.T; ++t) part[t * a.H] = ysum[t * z.rows + row];
      }
    }
  }
  meet<SHIFT>(sh, warp, ok, r, a.status);
  if (warp == kMulWarp<SHIFT>) tmem_free(sh.tmem, z.cols);
  if (z.slices == 2) {
    // The cluster's CTAs hold sums over their slices for the same columns of y
    // (one tile: the host cuts no more): each adds a share of them.
    __syncwarp();
    cluster_sync();
    const int64_t tiles = gridDim.x / z.slices, tile_id = blockIdx.x / z.slices;
    const int64_t r0 = a.H * tile_id / tiles;
    const int nr = (int)(a.H * (tile_id + 1) / tiles - r0), all = a.T * nr, slice = blockIdx.x % z.slices;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + r0;
    for (int i = all * slice / z.slices + threadIdx.x; i < all * (slice + 1) / z.slices; i += kStreamThreads<SHIFT>) {
      const int t = i / nr, row = i % nr;
      float sum = 0.0f;
      for (int k = 0; k < z.slices; ++k) sum += load_peer(ysum + t * z.rows + row, k);
      y[t * a.H + row] = __float2bfloat16_rn(sum);
    }
    __syncwarp();
    cluster_sync();  // nobody leaves while its sums are read
  }
}

// y = the sum of the slices' parts, in their order; four columns a thread.
__global__ void __launch_bounds__(kThreads)
    sum_parts_kernel(const float* __restrict__ parts, int64_t ld, int slices, int64_t n, __nv_bfloat16* __restrict__ y) {
  await_previous_kernel();
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
  if (i >= n) return;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int k = 0; k < slices; ++k) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(parts + k * ld + i));
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  y[i] = __float2bfloat16_rn(sum.x);
  if (i + 1 < n) y[i + 1] = __float2bfloat16_rn(sum.y);
  if (i + 2 < n) y[i + 2] = __float2bfloat16_rn(sum.z);
  if (i + 3 < n) y[i + 3] = __float2bfloat16_rn(sum.w);
}

// ------------------------------------------------------------------ host

// Elements of a row padded to 32 bytes (of fp32, what 16 bytes of bf16 weights go with).
int64_t padded_row(int64_t n) { return (n + 7) / 8 * 8; }

template <typename ET, bool SHIFT>
int run_router(const LayerArgs& a, const ET* x, int64_t x_ld, const void* router, float* logits, int32_t mode,
               int32_t normalize, int32_t* top_expert, float* weights, cudaStream_t s) {
  static std::atomic<bool> raised[kSmemDevices];
  auto r = router_rows_kernel<ET, SHIFT>;
  if (!allow_smem(r, raised)) return MOE_ERR_CUDA;
  launch(r, dim3((unsigned)((a.E + kRows - 1) / kRows), (unsigned)((a.T + kCols - 1) / kCols)), kThreads, kRowsRing<ET, SHIFT>, s, x, x_ld,
         static_cast<const ET*>(router), a.H, a.T, a.E, logits);
  return moe_topk_gating(logits, a.T, a.E, a.K, mode, normalize, top_expert, weights,
                         reinterpret_cast<moe_stream_t>(s));
}

template <typename ET, bool SHIFT> int run_rows(const LayerArgs& a, const ET* x, int64_t x_ld, cudaStream_t s) {
  static std::atomic<bool> raised_g[kSmemDevices], raised_d[kSmemDevices];
  const size_t seg = kRowsRing<ET, SHIFT> + segments_bytes(a.n, a.E);
  const int64_t h_ld = padded_row(a.F), couples = (a.F + 1) / 2;
  auto g = gate_up_rows_kernel<ET, SHIFT>;
  if (!allow_smem(g, raised_g)) return MOE_ERR_CUDA;
  launch(g, grid_for(g, kThreads, seg, ((a.n < a.E ? a.n : a.E) * couples + kWarps - 1) / kWarps), kThreads, seg, s, a, x,
         x_ld, h_ld);
  const size_t smem = seg + sizeof(int32_t) * a.n + sizeof(float) * kRows * a.n * (a.n <= kSliceChoices ? kWarps : 1);
  auto d = down_rows_kernel<ET, SHIFT>;
  if (!allow_smem(d, raised_d)) return MOE_ERR_CUDA;
  launch(d, grid_for(d, kThreads, smem, (a.H + kRows - 1) / kRows), kThreads, smem, s, a, h_ld);
  return check_launch();
}

// cuTensorMapEncodeTiled through the runtime (the library links no driver library).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static std::atomic<EncodeFn> cached{nullptr};
  EncodeFn f = cached.load(std::memory_order_relaxed);
  if (f != nullptr) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess) {
    (void)cudaGetLastError();
    return nullptr;
  }
  f = reinterpret_cast<EncodeFn>(p);
  cached.store(f, std::memory_order_relaxed);
  return f;
}

// bf16 [nz, ny, nx], contiguous, read in boxes of 64 x by x bz, swizzled by 128 bytes; what lies outside reads as zero.
bool tensor_map(CUtensorMap* map, const void* base, int64_t nx, int64_t ny, int64_t nz, int by, int bz) {
  const EncodeFn f = encode_fn();
  if (f == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)nx, (cuuint64_t)ny, (cuuint64_t)nz};
  const cuuint64_t strides[2] = {(cuuint64_t)nx * 2, (cuuint64_t)nx * ny * 2};
  const cuuint32_t box[3] = {kBlock, (cuuint32_t)by, (cuuint32_t)bz}, step[3] = {1, 1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxSms = 192;             // that the layer uses: bounds the workspace
constexpr int kSmBytes = 226 * 1024;  // dynamic shared memory of a CTA at most, beside its static part

// Stages of stage_bytes that fit beside `rest` bytes; false for fewer than two.
bool fit_stages(StreamShape* z, size_t rest) {
  const int64_t n = ((int64_t)kSmBytes - (int64_t)sizeof(StreamShared) - 1024 - (int64_t)rest) / z->stage_bytes;
  z->stages = (int)(n < kMaxStages ? n : kMaxStages);
  return n >= 2;
}
uint32_t tmem_cols(int cols) {
  uint32_t c = 32;
  while ((int)c < cols) c *= 2;
  return c;
}

// Blocks of a stage, `most` or as many fewer as leave `least` stages (two with one block).
template <bool SHIFT> bool cut_stages(StreamShape* z, int block_bytes, int most, size_t rest) {
  constexpr int least = SHIFT ? 2 : 3;
  for (z->blocks = most; z->blocks >= 1; --z->blocks) {
    z->stage_bytes = z->blocks * block_bytes;
    if (fit_stages(z, rest + (SHIFT ? raw_bytes(z->blocks) : 0)) && (z->stages >= least || z->blocks == 1)) return true;
  }
  return false;
}

template <bool SHIFT> int run_stream(const LayerArgs& a, float* parts, cudaStream_t s) {
  static std::atomic<bool> raised_g[kSmemDevices], raised_d[kSmemDevices];
  __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(a.h);
  const int64_t h_ld = padded_row(a.F), y_n = a.T * a.H, parts_ld = (y_n + 3) / 4 * 4;
  const StreamArgs p{a, h, h + a.n * h_ld, h_ld, parts, parts_ld, test_give_up().load(std::memory_order_relaxed)};
  const int64_t sms = num_sms() < kMaxSms ? num_sms() : kMaxSms;
  const size_t seg = segments_bytes(a.n, a.E);
  // Tokens of an expert at a time: twice the mean and 16, so that few experts
  // take a second pass over their weights and stages hold weights in the main.
  const int cap = 2 * a.n / a.E + 16 < kMaxTokens ? round_to(2 * a.n / a.E + 16, 16) : kMaxTokens;

  // Blocks of a stage: consecutive 128-byte pieces of a row, which the memory
  // delivers better the more there are (the first kernel's weights of the
  // Mixtral-8x7B shape, 8 tokens: 5.7 TB/s with one block, 6.6 with three; 64
  // rows and four blocks: 6.7, but 5.3 instead of 5.9 at one token).
  StreamShape g{};
  g.slices = 1;
  g.rows = kTileRows;
  g.tokens = round_to(a.T, 16) < cap ? round_to(a.T, 16) : cap;
  g.cols = tmem_cols(2 * g.tokens);
  if (!cut_stages<SHIFT>(&g, (g.rows + g.tokens) * kRowBytes, 3, seg)) return MOE_ERR_UNSUPPORTED;
  const size_t g_smem = seg + (size_t)g.stages * g.stage_bytes + (SHIFT ? raw_bytes(g.blocks) : 0) + 1024;

  // A product costs the same whatever rows of its 128 the tile holds (27 rows,
  // H 2048 over pairs of SMs: 2.3 TB/s), and every tile reads all of h. So
  // tiles have close to 128 rows, and as many SMs share one as there are for
  // it: each takes an equal share of the active experts' blocks, and the sums
  // meet in the pair's shared memory or, for more than two, in the workspace
  // and a kernel that adds them (16 tokens, 2048 x 768, 64 experts, 8 each:
  // 43 us and 3 instead of 78; 64 tokens, 1024 x 1024, 256 experts: 102 and 3
  // instead of 364). Stages of up to 64 KB, for the reason above: 48 tokens of
  // the Mixtral-8x22B shape 3.9 TB/s at 32 KB, 6.2 at 64.
  // Where the sums of all tokens leave the ring too little, an expert's tokens
  // take more passes first (64 at a time), then tiles get smaller.
  StreamShape d{};
  const int d_tokens = round_to(a.T, 8) < cap ? round_to(a.T, 8) : cap;
  int64_t grid = 0;
  size_t d_smem = 0;
  bool fits = false;
  for (int most = kTileRows; !fits && most >= 16; most /= 2) {
    const int64_t need = (a.H + most - 1) / most;
    d.slices = need < sms ? (int)(sms / need) : 1;
    const int64_t tiles = sms / d.slices < a.H ? sms / d.slices : a.H, share = (a.H + tiles - 1) / tiles;
    d.rows = (int)(share < most ? share : most);
    grid = tiles * d.slices;
    for (const int tokens : {d_tokens, d_tokens < 64 ? d_tokens : 64}) {
      if (fits) break;
      d.tokens = tokens;
      const int block = (round_to(d.rows, 8) + 2 * d.tokens) * kRowBytes;
      // A product reads 128 rows from a block's start whatever the tile holds:
      // behind the ring lie at least as many bytes of the CTA's memory.
      d_smem = seg + sizeof(float) * a.T * d.rows;
      if (d_smem < kTileRows * kRowBytes) d_smem = kTileRows * kRowBytes;
      fits = cut_stages<SHIFT>(&d, block, SHIFT ? 3 : block < 65536 ? 65536 / block : 1, d_smem);
    }
  }
  d.cols = tmem_cols(4 * d.tokens);
  if (!fits) return MOE_ERR_UNSUPPORTED;
  d_smem += (size_t)d.stages * d.stage_bytes + (SHIFT ? raw_bytes(d.blocks) : 0) + 1024;

  CUtensorMap g_map = {}, d_map = {};
  if (!allow_smem(gate_up_stream_kernel<SHIFT>, raised_g) ||
      !allow_smem(down_stream_kernel<SHIFT>, raised_d) ||
      (!SHIFT && (!tensor_map(&g_map, a.w_gate_up, a.H, a.F, 2 * (int64_t)a.E, 16, 2) ||
                  !tensor_map(&d_map, a.w_down, a.F, a.H, a.E, d.rows, 1))))
    return MOE_ERR_CUDA;
  const int64_t pairs = (a.n < a.E ? a.n : a.E) * a.F;
  launch(gate_up_stream_kernel<SHIFT>, (unsigned)(pairs < sms ? pairs : sms), kStreamThreads<SHIFT>, g_smem, s, p, g, g_map);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kStreamThreads<SHIFT>);
  cfg.dynamicSmemBytes = d_smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)d.slices, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = d.slices == 2 ? 2 : 1;
  (void)cudaLaunchKernelEx(&cfg, down_stream_kernel<SHIFT>, p, d, d_map);
  if (d.slices > 2)
    launch(sum_parts_kernel, (unsigned)((parts_ld / 4 + kThreads - 1) / kThreads), kThreads, 0, s, p.parts, parts_ld, d.slices, y_n,
           static_cast<__nv_bfloat16*>(a.y));
  return check_launch();
}

constexpr int64_t kSmallLayer = 1 << 24;

template <typename ET>
int dispatch(const LayerArgs& a, const void* router, float* logits, float* parts, ET* x_copy, int32_t mode, int32_t normalize,
             int32_t* top_expert, float* weights, cudaStream_t s) {
  constexpr int kE = 16 / Elem<ET>::kBytes;
  const ET* x = static_cast<const ET*>(a.x);
  int64_t x_ld = a.x_stride;
  if (a.H % kE != 0 || x_ld % kE != 0 || !aligned(a.x, 16)) {
    const int64_t padded = padded_row(a.H);
    launch(align_rows_kernel<ET>, dim3((unsigned)((padded + 4 * kThreads - 1) / (4 * kThreads)), (unsigned)a.T), kThreads, 0, s, x,
           x_ld, a.H, padded, x_copy);
    x = x_copy;
    x_ld = padded;
  }
  if (router != nullptr) {
    const int rc = a.H % kE == 0 && aligned(router, 16)
                       ? run_router<ET, false>(a, x, x_ld, router, logits, mode, normalize, top_expert, weights, s)
                       : run_router<ET, true>(a, x, x_ld, router, logits, mode, normalize, top_expert, weights, s);
    if (rc != MOE_OK) return rc;
  }
  const bool by16 = a.H % kE == 0 && a.F % kE == 0 && aligned(a.w_gate_up, 16) && aligned(a.w_down, 16);
  if constexpr (Elem<ET>::kBytes == 2) {
    // The tensor path costs some 8 us more to start: below 100 MB of weights
    // (every choice's own) the ordinary cores are ahead. One token, 512 x 512,
    // 2 of 8 experts: 10.8 us on these, 22.2 on tensor cores; 1024 x 2048:
    // 15.9 and 24.2; 4 tokens of it (100 MB): 31.3 and 31.5; 8: 39.1 and 35.3.
    // Many tokens to an expert are slow on them: 16 tokens, 512 x 512: 21 and
    // 24.6 us; 32 (8 an expert): 26.9 and 25.8.
    const bool small = a.n * a.H * a.F <= kSmallLayer && a.n <= 4 * a.E;
    if (a.H >= kBlock && a.F >= kBlock && !small) {  // at least one box each way
      LayerArgs b = a;
      b.x = x;
      b.x_stride = x_ld;
      return by16 ? run_stream<false>(b, parts, s) : run_stream<true>(b, parts, s);
    }
  }
  if (!by16) return run_rows<ET, true>(a, x, x_ld, s);
  return run_rows<ET, false>(a, x, x_ld, s);
}

// Bytes of the workspace's parts: the logits, h, the slices' sums of y, and x where its rows are not aligned.
size_t logits_bytes(int64_t T, int32_t E) { return ((size_t)T * E * sizeof(float) + 255) / 256 * 256; }
size_t h_bytes(int64_t n, int64_t F) { return ((size_t)n * (size_t)padded_row(F) * sizeof(float) + 255) / 256 * 256; }

// slices * H <= SMs * the rows of a tile, and a tile has no more rows than y columns.
size_t parts_bytes(int64_t T, int64_t H) { return kMaxSms * ((size_t)T * (H < kTileRows ? H : kTileRows) + 4) * sizeof(float); }

bool sizes_ok(int64_t T, int64_t H, int64_t F, int32_t E, int32_t K) {
  return T >= 0 && H >= 1 && F >= 1 && E >= 1 && K >= 1 && K <= E && K <= MOE_MAX_TOP_K &&
         H <= INT32_MAX / 2 && F <= INT32_MAX / 4 && H <= INT64_MAX / 16 / F / E;
}
bool few(int64_t T, int32_t E, int32_t K) {
  return E <= MOE_GATING_MAX_EXPERTS && T <= MOE_LAYER_MAX_TOKENS && T * K <= MOE_LAYER_MAX_CHOICES;
}

int run_layer(const void* x, int32_t dtype, int64_t x_stride, const void* router, const void* w_gate_up,
              const void* w_down, int64_t T, int64_t H, int64_t F, int32_t E, int32_t K, int32_t mode,
              int32_t normalize, int32_t* top_out, float* weights_out, const int32_t* top_expert,
              const float* weights, void* y, void* workspace, size_t workspace_bytes, int32_t* d_status,
              moe_stream_t stream) {
  if (!sizes_ok(T, H, F, E, K)) return MOE_ERR_INVALID_ARG;
  const int eb = dtype_bytes(dtype);
  if (eb == 0 || !few(T, E, K)) return MOE_ERR_UNSUPPORTED;
  if (T > 1 && (x_stride < H || x_stride > INT64_MAX / 16 / T)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (x == nullptr || w_gate_up == nullptr || w_down == nullptr || top_expert == nullptr || weights == nullptr ||
      y == nullptr || workspace == nullptr || workspace_bytes < moe_layer_workspace_size(T, H, F, E, K))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, eb) || !aligned(router, eb) || !aligned(w_gate_up, eb) || !aligned(w_down, eb) || !aligned(y, eb) ||
      !aligned(top_expert, 4) || !aligned(weights, 4) || !aligned(workspace, 16) || !aligned(d_status, 4))
    return MOE_ERR_UNSUPPORTED;
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~(uintptr_t)255);
  float* logits = reinterpret_cast<float*>(base);
  float* h = reinterpret_cast<float*>(base + logits_bytes(T, E));
  const LayerArgs a{x, w_gate_up, w_down, top_expert, weights, h, y, T > 1 ? x_stride : H, H, F,
                    (int32_t)T, E, K, (int32_t)(T * K), d_status};
  float* parts = reinterpret_cast<float*>(reinterpret_cast<char*>(h) + h_bytes(T * K, F));
  void* x_copy = reinterpret_cast<char*>(parts) + parts_bytes(T, H);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MOE_F32)
    return dispatch<float>(a, router, logits, parts, static_cast<float*>(x_copy), mode, normalize, top_out, weights_out, s);
  return dispatch<__nv_bfloat16>(a, router, logits, parts, static_cast<__nv_bfloat16*>(x_copy), mode, normalize, top_out,
                                 weights_out, s);
}

}  // namespace

std::atomic<uint32_t>& test_give_up() {
  static std::atomic<uint32_t> bits{0};
  return bits;
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_layer_workspace_size(int64_t T, int64_t H, int64_t F, int32_t E, int32_t K) {
  if (!sizes_ok(T, H, F, E, K) || !few(T, E, K)) return 0;
  return logits_bytes(T, E) + h_bytes(T * K, F) + parts_bytes(T, H) + (size_t)T * (size_t)padded_row(H) * sizeof(float) + 256;
}

extern "C" int moe_layer(const void* x, int32_t dtype, int64_t x_stride, const void* router, const void* w_gate_up,
                         const void* w_down, int64_t T, int64_t H, int64_t F, int32_t E, int32_t K, int32_t mode,
                         int32_t normalize, int32_t* top_expert, float* weights, void* y, void* workspace,
                         size_t workspace_bytes, int32_t* d_status, moe_stream_t stream) {
  if (mode != MOE_GATING_SOFTMAX && mode != MOE_GATING_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (T > 0 && router == nullptr) return MOE_ERR_INVALID_ARG;
  return run_layer(x, dtype, x_stride, router, w_gate_up, w_down, T, H, F, E, K, mode, normalize, top_expert, weights,
                   top_expert, weights, y, workspace, workspace_bytes, d_status, stream);
}

extern "C" int moe_experts(const void* x, int32_t dtype, int64_t x_stride, const int32_t* top_expert,
                           const float* weights, const void* w_gate_up, const void* w_down, int64_t T, int64_t H,
                           int64_t F, int32_t E, int32_t K, void* y, void* workspace, size_t workspace_bytes,
                           int32_t* d_status, moe_stream_t stream) {
  return run_layer(x, dtype, x_stride, nullptr, w_gate_up, w_down, T, H, F, E, K, 0, 0, nullptr, nullptr, top_expert,
                   weights, y, workspace, workspace_bytes, d_status, stream);
}

extern "C" void moe_test_block_waits(uint32_t give_up) { test_give_up().store(give_up, std::memory_order_relaxed); }
