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

// ------------------------------------------------------- choices by expert

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

// Called by the whole CTA; warp 0 does the work.
__device__ __forceinline__ Segments sort_choices(const int32_t* __restrict__ top_expert, int32_t n, int32_t E, int32_t K,
                                                 int32_t* status, int32_t* smem) {
  const int m = n < E ? n : E;
  Segments s;
  s.order = smem;
  s.token = smem + n;
  int32_t* local = s.token + n;  // rank of an assignment within its expert
  int32_t* count = local + n;  // [E]: choices of the expert, then where they begin
  s.expert = count + E;
  s.begin = s.expert + m;
  int32_t* active = s.begin + m + 1;
  const int lane = lane_id();
  if (threadIdx.x < kWarp) {
    for (int e = lane; e < E; e += kWarp) count[e] = 0;
    __syncwarp();
    for (int i0 = 0; i0 < n; i0 += kWarp) {
      const int i = i0 + lane;
      int e = i < n ? __ldcg(top_expert + i) : -1;
      if (e < -1 || e >= E) {
        if (blockIdx.x == 0) flag_status(status, MOE_STATUS_BAD_EXPERT);
        e = -1;
      }
      const unsigned peers = __match_any_sync(0xffffffffu, e);
      if (e >= 0) local[i] = count[e] + __popc(peers & lanemask_lt());
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
    __syncwarp();
    for (int i = lane; i < n; i += kWarp) {
      const int e = __ldcg(top_expert + i);
      if (e < 0 || e >= E) continue;
      const int at = count[e] + local[i];
      s.order[at] = i;
      s.token[at] = i / K;
    }
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
// A warp per weight row: its lanes stride over the row in vectors of VB
// bytes (the widest that the lengths and addresses allow), kCols tokens at a
// time, in fp32. Takes fp32 layers and rows that are not a multiple of 16 bytes.

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / kWarp;
constexpr int kCols = 4;

template <int VB, typename ET>
__global__ void __launch_bounds__(kThreads)
    router_rows_kernel(const void* __restrict__ x, int64_t x_stride, const void* __restrict__ router, int64_t H, int32_t T,
                       int32_t E, float* __restrict__ logits) {
  using L = Lanes<VB, ET>;
  using V = typename L::V;
  await_previous_kernel();
  const int lane = lane_id();
  const int tiles = (T + kCols - 1) / kCols;
  const int64_t vecs = H / L::kElems;
  for (int64_t w = (int64_t)blockIdx.x * kWarps + threadIdx.x / kWarp; w < (int64_t)tiles * E;
       w += (int64_t)gridDim.x * kWarps) {
    const int e = (int)(w % E), t0 = (int)(w / E) * kCols;
    const V* r = reinterpret_cast<const V*>(static_cast<const ET*>(router) + e * H);
    const V* px[kCols];
    float acc[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      const int t = t0 + c < T ? t0 + c : T - 1;
      px[c] = reinterpret_cast<const V*>(static_cast<const ET*>(x) + t * x_stride);
      acc[c] = 0.0f;
    }
#pragma unroll 2
    for (int64_t i = lane; i < vecs; i += kWarp) {
      const V rv = ld_l1(r + i);
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const V xv = ld_l1(px[c] + i);
#pragma unroll
        for (int q = 0; q < L::kElems; ++q) acc[c] += L::get(rv, q) * L::get(xv, q);
      }
    }
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      const float s = warp_sum(acc[c]);
      if (lane == 0 && t0 + c < T) logits[(int64_t)(t0 + c) * E + e] = s;
    }
  }
}

template <int VB, typename ET> __global__ void __launch_bounds__(kThreads) gate_up_rows_kernel(LayerArgs a) {
  using L = Lanes<VB, ET>;
  using V = typename L::V;
  extern __shared__ int32_t smem[];
  await_previous_kernel();
  const Segments s = sort_choices(a.top_expert, a.n, a.E, a.K, a.status, smem);
  const int lane = lane_id();
  const int64_t vecs = a.H / L::kElems;
  for (int64_t w = (int64_t)blockIdx.x * kWarps + threadIdx.x / kWarp; w < s.active * a.F;
       w += (int64_t)gridDim.x * kWarps) {
    const int q = (int)(w / a.F);
    const int64_t f = w % a.F;
    const ET* gate = static_cast<const ET*>(a.w_gate_up) + ((int64_t)s.expert[q] * 2 * a.F + f) * a.H;
    const V* pg = reinterpret_cast<const V*>(gate);
    const V* pu = reinterpret_cast<const V*>(gate + a.F * a.H);
    for (int i0 = s.begin[q]; i0 < s.begin[q + 1]; i0 += kCols) {
      const int last = s.begin[q + 1] - 1;
      const V* px[kCols];
      float g[kCols], u[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const int t = s.token[i0 + c < last ? i0 + c : last];
        px[c] = reinterpret_cast<const V*>(static_cast<const ET*>(a.x) + t * a.x_stride);
        g[c] = u[c] = 0.0f;
      }
#pragma unroll 2
      for (int64_t i = lane; i < vecs; i += kWarp) {
        const V gv = ld_l1(pg + i), uv = ld_l1(pu + i);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const V xv = ld_l1(px[c] + i);
#pragma unroll
          for (int k = 0; k < L::kElems; ++k) {
            g[c] += L::get(gv, k) * L::get(xv, k);
            u[c] += L::get(uv, k) * L::get(xv, k);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const float gs = warp_sum(g[c]), us = warp_sum(u[c]);
        if (lane == 0 && i0 + c <= last) a.h[(i0 + c) * a.F + f] = a.weights[s.order[i0 + c]] * (silu(gs) * us);
      }
    }
  }
}

template <int VB, typename ET> __global__ void __launch_bounds__(kThreads) down_rows_kernel(LayerArgs a) {
  using L = Lanes<VB, ET>;
  using V = typename L::V;
  extern __shared__ int32_t smem[];
  await_previous_kernel();
  const Segments s = sort_choices(a.top_expert, a.n, a.E, a.K, a.status, smem);
  const int lane = lane_id();
  // This warp's row of y for every token.
  float* sum = reinterpret_cast<float*>(smem + segments_bytes(a.n, a.E) / sizeof(int32_t)) +
               (threadIdx.x / kWarp) * a.T;
  const int64_t vecs = a.F / L::kElems;
  for (int64_t r = (int64_t)blockIdx.x * kWarps + threadIdx.x / kWarp; r < a.H; r += (int64_t)gridDim.x * kWarps) {
    for (int t = lane; t < a.T; t += kWarp) sum[t] = 0.0f;
    __syncwarp();
    for (int q = 0; q < s.active; ++q) {
      const V* pw = reinterpret_cast<const V*>(static_cast<const ET*>(a.w_down) + ((int64_t)s.expert[q] * a.H + r) * a.F);
      const int last = s.begin[q + 1] - 1;
      for (int i0 = s.begin[q]; i0 <= last; i0 += kCols) {
        const float* ph[kCols];
        float acc[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          ph[c] = a.h + (i0 + c < last ? i0 + c : last) * a.F;
          acc[c] = 0.0f;
        }
#pragma unroll 2
        for (int64_t i = lane; i < vecs; i += kWarp) {
          const V wv = ld_l1(pw + i);
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
#pragma unroll
            for (int k = 0; k < L::kElems; ++k) acc[c] += L::get(wv, k) * __ldg(ph[c] + i * L::kElems + k);
          }
        }
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const float v = warp_sum(acc[c]);
          if (lane == 0 && i0 + c <= last) sum[s.token[i0 + c]] += v;
        }
      }
    }
    __syncwarp();
    for (int t = lane; t < a.T; t += kWarp) {
      if constexpr (Elem<ET>::kBytes == 4)
        static_cast<float*>(a.y)[t * a.H + r] = sum[t];
      else
        static_cast<__nv_bfloat16*>(a.y)[t * a.H + r] = __float2bfloat16_rn(sum[t]);
    }
    __syncwarp();
  }
}

// ------------------------------------------------- bf16 rows of 16 bytes
//
// Weights stream through a ring of shared-memory stages and are multiplied by
// eight consumer warps with m16n8k16 tensor instructions: 16 weight rows by 8
// tokens, an expert's tokens in up to NT such tiles. With few tokens the time
// is that of the weight bytes, so what matters is that copies are always in
// flight: the copying warps run ahead of the consumers across tiles, rows and
// experts, and the work is cut so that each of the SMs streams the same number
// of bytes (an equal share of the active experts' F gate/up row pairs; an
// equal share of y's H columns for all experts), whatever the sizes.
//
// The weights come by tensor copies (TMA), one thread's work: 4 KB and more
// an instruction. The same ring filled with bulk copies of 1 KB pieces of rows
// reached 4.5 TB/s (an SM starts one in 34 ns whatever its size), with 16-byte
// asynchronous copies of four warps 5 TB/s (their instructions), with tensor
// copies of 64 elements by 32 rows 7.0 TB/s. The tokens' rows, which lie
// apart, come by 16-byte copies of kTokenWarps warps.
//
// A stage holds nb blocks of 64 elements: first the weights, block by block,
// each row's 128 bytes with the 16-byte pieces exchanged by the copy's 128-byte
// swizzle, then the tokens' rows, nb * 128 + 16 bytes apart. Lane (g, c) of a
// warp reads pieces 2c and 2c + 1 of rows g and g + 8 and of token g: no bank
// conflicts on either side. A piece feeds two instructions; that pairs k's in
// another order than the instruction's own, on both sides alike, which a dot
// product does not see. The warps share a stage's tile, MT tiles of 16 rows by
// KS slices of the blocks, and add their sums in shared memory at the tile's
// end, in a fixed order.

constexpr int kConsumers = 8;
constexpr int kTokenWarps = 3;
constexpr int kCopyWarp = kConsumers + kTokenWarps;  // the warp that copies weights
constexpr int kStreamThreads = (kCopyWarp + 1) * kWarp;
constexpr int kStages = 3;
constexpr int kBlock = 64;  // elements of a block: the 128 bytes of a swizzled row

__host__ __device__ constexpr int k_slices(int MT) { return MT == 4 ? 2 : 4; }
// Bytes of a stage of nb blocks, and the blocks that fit (not 0: the host
// chooses stages and tokens at a time that hold one). Swizzled blocks start
// on 1 KB boundaries.
__host__ __device__ inline int block_bytes(int rows) { return (rows + 7) / 8 * 1024; }
__host__ __device__ inline int stage_blocks(int stage_bytes, int wrows, int trows) {
  return (stage_bytes - 16 * trows) / (block_bytes(wrows) + 2 * kBlock * trows);
}

__device__ __forceinline__ void mbar_init_count(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// Lets the next kernel on the stream start while this one runs.
__device__ __forceinline__ void allow_next_kernel() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A box of the tensor from coordinates (x, y, z); x is a multiple of 64.
__device__ __forceinline__ void tensor_copy(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2,%3,%4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// 16 bytes from global to shared memory, not through L1.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The thread's arrival on the barrier, once all its copies so far have landed.
__device__ __forceinline__ void arrive_after_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
  return v;
}
// d += A (16 rows x 16) * B (16 x 8), bf16 operands, fp32 sums.
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The ring's barriers and where one side stands in it.
struct Ring {
  uint32_t data, full, empty;  // shared-memory addresses
  int stage_bytes;
  int stage;
  uint32_t parity;
  bool ok;  // false after a wait gave up: nothing is waited for or copied any more
  __device__ __forceinline__ uint32_t at() const { return data + stage * stage_bytes; }
  __device__ __forceinline__ uint32_t full_bar() const { return full + 8 * stage; }
  // By a whole warp; bounded.
  __device__ __forceinline__ void wait(uint32_t bars, int32_t* status) {
    if (!ok) return;
    ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * stage, parity));
    if (!ok && lane_id() == 0) flag_status(status, MOE_STATUS_TIMEOUT);
  }
  __device__ __forceinline__ void advance() {
    if (++stage == kStages) {
      stage = 0;
      parity ^= 1;
    }
  }
};

__device__ __forceinline__ Ring make_ring(uint32_t data, uint32_t bars, int stage_bytes, bool copies) {
  // A copying warp's first wait on each stage passes: a fresh barrier counts as one phase done.
  return Ring{data, bars, bars + 8 * kStages, stage_bytes, 0, copies ? 1u : 0u, true};
}
__device__ __forceinline__ void init_ring(uint32_t bars) {
  for (int i = 0; i < kStages; ++i) {
    mbar_init_count(bars + 8 * i, kTokenWarps * kWarp + 1);
    mbar_init_count(bars + 8 * (kStages + i), kConsumers);
  }
  fence_mbarrier_init();
}
__device__ __forceinline__ uint32_t align_1k(uint32_t p) { return (p + 1023u) & ~1023u; }

// Adds one stage's products to acc: this warp's blocks (ks, ks + KS, ...), of
// which weight rows row0 and row1 (this lane's two of 16) and the tokens at
// tok. kc: elements of the stage; beyond them the weights are zero and the
// tokens' places are taken as zero. PARTS 2: the tokens' rows are held as the
// sum of two bf16 numbers, the second ntok rows after the first.
template <int NT, int PARTS, int KS, int TILES>
__device__ __forceinline__ void multiply_tiles(float (&acc)[NT][4], uint32_t weights, int block, int kc, int ks,
                                               int row0, int row1, uint32_t tok, int tok_stride, int ntok) {
  const int lane = lane_id(), g = lane >> 2, c = lane & 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // One tile: a second set of sums, so that an instruction does not wait for the one before it.
  float odd[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  uint32_t at[TILES];
#pragma unroll
  for (int j = 0; j < TILES; ++j) at[j] = tok + (uint32_t)(j * 8 + g < ntok ? j * 8 + g : ntok - 1) * tok_stride + c * 32;
  const uint32_t p0 = weights + row0 * 128, p1 = weights + row1 * 128;
  for (int b = ks; b * kBlock < kc; b += KS) {
    uint4 a0[2], a1[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      a0[s] = lds16(p0 + b * block + (((2 * c + s) ^ (row0 & 7)) << 4));
      a1[s] = lds16(p1 + b * block + (((2 * c + s) ^ (row1 & 7)) << 4));
    }
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bool in = b * kBlock + (2 * c + s) * 8 < kc;
        uint4 v[TILES];
#pragma unroll
        for (int j = 0; j < TILES; ++j) v[j] = in ? lds16(at[j] + p * ntok * tok_stride + b * 2 * kBlock + s * 16) : zero;
#pragma unroll
        for (int j = 0; j < TILES; ++j) mma16(acc[j], a0[s].x, a1[s].x, a0[s].y, a1[s].y, v[j].x, v[j].y);
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
          if (TILES == 1)
            mma16(odd, a0[s].z, a1[s].z, a0[s].w, a1[s].w, v[j].z, v[j].w);
          else
            mma16(acc[j], a0[s].z, a1[s].z, a0[s].w, a1[s].w, v[j].z, v[j].w);
        }
      }
    }
  }
  if (TILES == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[0][i] += odd[i];
  }
}

template <int NT, int PARTS, int KS>
__device__ __forceinline__ void multiply_stage(float (&acc)[NT][4], uint32_t weights, int block, int kc, int ks,
                                               int row0, int row1, uint32_t tok, int tok_stride, int ntok) {
  if (NT == 1 || ntok <= 8)
    multiply_tiles<NT, PARTS, KS, 1>(acc, weights, block, kc, ks, row0, row1, tok, tok_stride, ntok);
  else if (NT == 2 || ntok <= 16)
    multiply_tiles<NT, PARTS, KS, NT < 2 ? NT : 2>(acc, weights, block, kc, ks, row0, row1, tok, tok_stride, ntok);
  else if (NT > 3 && ntok <= 24)
    multiply_tiles<NT, PARTS, KS, NT < 3 ? NT : 3>(acc, weights, block, kc, ks, row0, row1, tok, tok_stride, ntok);
  else if (NT == 4 || ntok <= 32)
    multiply_tiles<NT, PARTS, KS, NT < 4 ? NT : 4>(acc, weights, block, kc, ks, row0, row1, tok, tok_stride, ntok);
  else
    multiply_tiles<NT, PARTS, KS, NT>(acc, weights, block, kc, ks, row0, row1, tok, tok_stride, ntok);
}

// A warp's 16 x 8 sums, row-major, for the threads that add the KS slices.
__device__ __forceinline__ void put_tile(float* red, const float (&acc)[4]) {
  const int lane = lane_id();
  float* p = red + (lane >> 2) * 8 + (lane & 3) * 2;
  p[0] = acc[0];
  p[1] = acc[1];
  p[64] = acc[2];
  p[65] = acc[3];
}

struct StreamArgs {
  LayerArgs a;
  __nv_bfloat16* h_hi;  // [n, F] in sorted order: h = h_hi + h_lo
  __nv_bfloat16* h_lo;
  int stage_bytes;
  int gate_tokens, down_tokens;  // of an expert at a time: NT * 8, or fewer where a stage would not hold their rows
  int down_rows;                 // rows of a box of w_down
};

// Tiles of up to 16 row pairs (gate, up) of one expert by up to per_pass of
// its tokens, over the whole of H. A box always has 16 pairs: those beyond a
// CTA's share are read too (from L2, their owner reads them as well) and left.
struct GateUpWalk {
  const Segments& s;
  int64_t pos, end, F;
  int q, nf, i0, ntok, K, nb, k0, stage_bytes, per_pass;
  int64_t f0;
  __device__ GateUpWalk(const Segments& s_, const StreamArgs& p)
      : s(s_), F(p.a.F), K((int)p.a.H), stage_bytes(p.stage_bytes), per_pass(p.gate_tokens) {
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
    nf = m < 16 ? (int)m : 16;
    i0 = s.begin[q];
    pass();
  }
  __device__ __forceinline__ void pass() {
    const int left = s.begin[q + 1] - i0;
    ntok = left < per_pass ? left : per_pass;
    nb = stage_blocks(stage_bytes, 32, ntok);
    k0 = 0;
  }
  __device__ __forceinline__ int kc() const { return K - k0 < nb * kBlock ? K - k0 : nb * kBlock; }
  __device__ __forceinline__ bool last_stage() const { return k0 + nb * kBlock >= K; }
  __device__ __forceinline__ void next() {
    k0 += nb * kBlock;
    if (k0 < K) return;
    i0 += ntok;
    if (i0 < s.begin[q + 1]) return pass();
    pos += nf;
    if (pos < end) tile();
  }
};

template <int NT>
__global__ void __launch_bounds__(kStreamThreads, NT <= 2 ? 2 : 1)
    gate_up_stream_kernel(StreamArgs p, const __grid_constant__ CUtensorMap map) {
  extern __shared__ __align__(1024) unsigned char dyn[];
  __shared__ uint64_t bars[2 * kStages];
  __shared__ float red[kConsumers * 128];
  constexpr int kWeights = 32;  // weight rows of a stage: 16 gate rows, then 16 up rows
  const LayerArgs& a = p.a;
  await_previous_kernel();
  if (threadIdx.x == kStreamThreads - 1) init_ring(smem_u32(bars));
  const uint32_t ring = align_1k(smem_u32(dyn));
  const Segments s = sort_choices(a.top_expert, a.n, a.E, a.K, a.status,
                                  reinterpret_cast<int32_t*>(dyn + (ring - smem_u32(dyn)) + (size_t)kStages * p.stage_bytes));
  allow_next_kernel();
  const int warp = threadIdx.x / kWarp, lane = lane_id();
  GateUpWalk w(s, p);
  Ring r = make_ring(ring, smem_u32(bars), p.stage_bytes, warp >= kConsumers);
  if (warp == kCopyWarp) {
    for (; w.more(); w.next(), r.advance()) {
      r.wait(r.empty, a.status);
      if (!r.ok) break;
      if (lane == 0) {
        const int n = (w.kc() + kBlock - 1) / kBlock, z = 2 * s.expert[w.q];
        mbar_expect(r.full_bar(), n * block_bytes(kWeights));
        for (int b = 0; b < n; ++b)
          tensor_copy(r.at() + b * block_bytes(kWeights), &map, w.k0 + b * kBlock, (int)w.f0, z, r.full_bar());
      }
    }
    return;
  }
  if (warp >= kConsumers) {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x);
    for (; w.more(); w.next(), r.advance()) {
      r.wait(r.empty, a.status);
      if (!r.ok) break;
      const uint32_t tok = r.at() + w.nb * block_bytes(kWeights);
      const int stride = w.nb * 2 * kBlock + 16, kc = w.kc();
      for (int i = warp - kConsumers; i < w.ntok; i += kTokenWarps) {
        const __nv_bfloat16* src = x + s.token[w.i0 + i] * a.x_stride + w.k0;
        for (int c = lane * 8; c < kc; c += kWarp * 8) copy16(tok + i * stride + c * 2, src + c);
      }
      arrive_after_copies(r.full_bar());
    }
    return;
  }
  // Warps 0..3: slices of the gate rows; 4..7: of the up rows.
  constexpr int KS = k_slices(2);
  const int mt = warp / KS, ks = warp % KS, row = mt * 16 + (lane >> 2);
  while (w.more()) {
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
    const int nf = w.nf, i0 = w.i0, ntok = w.ntok;
    const int64_t f0 = w.f0;
    for (bool last = false; !last; w.next(), r.advance()) {
      last = w.last_stage();
      r.wait(r.full, a.status);
      if (r.ok)
        multiply_stage<NT, 1, KS>(acc, r.at(), block_bytes(kWeights), w.kc(), ks, row, row + 8,
                                  r.at() + w.nb * block_bytes(kWeights), w.nb * 2 * kBlock + 16, ntok);
      __syncwarp();
      if (lane == 0) mbar_arrive(r.empty + 8 * r.stage);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j * 8 >= ntok) break;
      put_tile(red + warp * 128, acc[j]);
      consumers_sync();
      const int f = threadIdx.x & 15, c = threadIdx.x >> 4;
      if (threadIdx.x < 128 && f < nf && j * 8 + c < ntok) {
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          g += red[k * 128 + f * 8 + c];
          u += red[(KS + k) * 128 + f * 8 + c];
        }
        const int i = i0 + j * 8 + c;
        const float h = __ldcg(a.weights + s.order[i]) * (silu(g) * u);
        // Two bf16 numbers keep 16 significant bits of h: one would round the layer's result twice.
        const __nv_bfloat16 hi = __float2bfloat16_rn(h);
        const float rest = h - __bfloat162float(hi);
        const int64_t at = i * a.F + f0 + f;
        p.h_hi[at] = hi;
        p.h_lo[at] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.0f);
      }
      consumers_sync();
    }
  }
}

// y's columns [r0, r0 + nr) for one expert's tokens after another, over the whole of F.
template <int MT> struct DownWalk {
  const Segments& s;
  int64_t r0, end;
  int nr, box, q, i0, ntok, K, nb, k0, stage_bytes, per_pass;
  __device__ DownWalk(const Segments& s_, const StreamArgs& p)
      : s(s_), box(p.down_rows), K((int)p.a.F), stage_bytes(p.stage_bytes), per_pass(p.down_tokens) {
    r0 = p.a.H * blockIdx.x / gridDim.x;
    end = p.a.H * (blockIdx.x + 1) / gridDim.x;
    if (s.active == 0) r0 = end;
    if (more()) tile();
  }
  __device__ __forceinline__ bool more() const { return r0 < end; }
  __device__ __forceinline__ void tile() {
    nr = end - r0 < box ? (int)(end - r0) : box;
    q = 0;
    i0 = 0;
    pass();
  }
  __device__ __forceinline__ void pass() {
    const int left = s.begin[q + 1] - i0;
    ntok = left < per_pass ? left : per_pass;
    nb = stage_blocks(stage_bytes, box, 2 * ntok);
    k0 = 0;
  }
  __device__ __forceinline__ int kc() const { return K - k0 < nb * kBlock ? K - k0 : nb * kBlock; }
  __device__ __forceinline__ bool last_stage() const { return k0 + nb * kBlock >= K; }
  __device__ __forceinline__ void next() {
    k0 += nb * kBlock;
    if (k0 < K) return;
    i0 += ntok;
    if (i0 < s.begin[q + 1]) return pass();
    if (++q < s.active) return pass();
    r0 += nr;
    if (r0 < end) tile();
  }
};

template <int NT, int MT>
__global__ void __launch_bounds__(kStreamThreads, NT <= 2 ? 2 : 1)
    down_stream_kernel(StreamArgs p, const __grid_constant__ CUtensorMap map) {
  extern __shared__ __align__(1024) unsigned char dyn[];
  __shared__ uint64_t bars[2 * kStages];
  __shared__ float red[kConsumers * 128];
  const LayerArgs& a = p.a;
  // The gate/up kernel has waited for all before it, so the routing may be
  // read and weights copied while it still runs; h may not.
  if (threadIdx.x == kStreamThreads - 1) init_ring(smem_u32(bars));
  const uint32_t ring = align_1k(smem_u32(dyn));
  int32_t* seg = reinterpret_cast<int32_t*>(dyn + (ring - smem_u32(dyn)) + (size_t)kStages * p.stage_bytes);
  const Segments s = sort_choices(a.top_expert, a.n, a.E, a.K, nullptr, seg);
  float* ysum = reinterpret_cast<float*>(seg + segments_bytes(a.n, a.E) / sizeof(int32_t));  // [T, nr]
  const int warp = threadIdx.x / kWarp, lane = lane_id();
  DownWalk<MT> w(s, p);
  Ring r = make_ring(ring, smem_u32(bars), p.stage_bytes, warp >= kConsumers);
  const int block = block_bytes(p.down_rows);
  if (warp == kCopyWarp) {
    for (; w.more(); w.next(), r.advance()) {
      r.wait(r.empty, a.status);
      if (!r.ok) break;
      if (lane == 0) {
        const int n = (w.kc() + kBlock - 1) / kBlock;
        mbar_expect(r.full_bar(), n * p.down_rows * 2 * kBlock);
        for (int b = 0; b < n; ++b)
          tensor_copy(r.at() + b * block, &map, w.k0 + b * kBlock, (int)w.r0, s.expert[w.q], r.full_bar());
      }
    }
    return;
  }
  if (warp >= kConsumers) {
    await_previous_kernel();
    for (; w.more(); w.next(), r.advance()) {
      r.wait(r.empty, a.status);
      if (!r.ok) break;
      const uint32_t tok = r.at() + w.nb * block;
      const int stride = w.nb * 2 * kBlock + 16, kc = w.kc();
      for (int i = warp - kConsumers; i < 2 * w.ntok; i += kTokenWarps) {
        const __nv_bfloat16* src = (i < w.ntok ? p.h_hi + (w.i0 + i) * a.F : p.h_lo + (w.i0 + i - w.ntok) * a.F) + w.k0;
        for (int c = lane * 8; c < kc; c += kWarp * 8) copy16(tok + i * stride + c * 2, src + c);
      }
      arrive_after_copies(r.full_bar());
    }
    return;
  }
  constexpr int KS = k_slices(MT);
  const int mt = warp / KS, ks = warp % KS, row = mt * 16 + (lane >> 2);
  int64_t r0 = a.H * blockIdx.x / gridDim.x;
  const int64_t r_end = a.H * (blockIdx.x + 1) / gridDim.x;
  for (; r0 < r_end; r0 += p.down_rows) {
    const int nr = r_end - r0 < p.down_rows ? (int)(r_end - r0) : p.down_rows;
    for (int i = threadIdx.x; i < a.T * nr; i += kConsumers * kWarp) ysum[i] = 0.0f;
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
    while (w.more() && w.r0 == r0) {
      const int i0 = w.i0, ntok = w.ntok;
      for (bool last = false; !last; w.next(), r.advance()) {
        last = w.last_stage();
        r.wait(r.full, a.status);
        if (r.ok && mt * 16 < nr)  // rows beyond nr repeat its last
          multiply_stage<NT, 2, KS>(acc, r.at(), block, w.kc(), ks, row < nr ? row : nr - 1,
                                    row + 8 < nr ? row + 8 : nr - 1, r.at() + w.nb * block, w.nb * 2 * kBlock + 16,
                                    ntok);
        __syncwarp();
        if (lane == 0) mbar_arrive(r.empty + 8 * r.stage);
      }
      // One token's experts one after another need no sum in between.
      if (ntok == 1 && w.more() && w.r0 == r0 && w.ntok == 1 && s.token[w.i0] == s.token[i0]) continue;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (j * 8 >= ntok) break;
        consumers_sync();  // the last tile's sums (or the zeros above) are done with
        if (mt < MT) put_tile(red + warp * 128, acc[j]);
        consumers_sync();
        for (int i = threadIdx.x; i < MT * 128; i += kConsumers * kWarp) {
          const int rr = (i >> 7) * 16 + ((i & 127) >> 3), c = i & 7;
          if (rr >= nr || j * 8 + c >= ntok) continue;
          const int* o = s.token + i0 + j * 8;
          const int t = o[c];
          if (c > 0 && o[c - 1] == t) continue;  // a token that chose an expert twice: its first column adds both
          float sum = ysum[t * nr + rr];
          for (int c2 = c; c2 < 8 && j * 8 + c2 < ntok && o[c2] == t; ++c2) {
#pragma unroll
            for (int k = 0; k < KS; ++k) sum += red[((i >> 7) * KS + k) * 128 + (i & 127) + c2 - c];
          }
          ysum[t * nr + rr] = sum;
        }
      }
      // All of them: multiply_stage may have rounded the number of tiles up.
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
    }
    consumers_sync();
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + r0;
    for (int i = threadIdx.x; i < a.T * nr; i += kConsumers * kWarp) {
      const int t = i / nr, rr = i - t * nr;
      y[t * a.H + rr] = __float2bfloat16_rn(ysum[i]);
    }
    consumers_sync();
  }
}

// Raises a kernel's dynamic shared memory limit once per device.
template <typename Kernel> bool allow_smem(Kernel k, int bytes, std::atomic<int>* granted) {
  int dev = 0;
  (void)cudaGetDevice(&dev);
  const bool cached = dev >= 0 && dev < 64;
  if (cached && granted[dev].load(std::memory_order_relaxed) >= bytes) return true;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  if (cached) granted[dev].store(bytes, std::memory_order_relaxed);
  return true;
}

// ------------------------------------------------------------------ host

template <int VB, typename ET>
int run_router(const LayerArgs& a, const void* router, float* logits, int32_t mode, int32_t normalize,
               int32_t* top_expert, float* weights, cudaStream_t s) {
  if (router == nullptr) return MOE_OK;
  auto k = router_rows_kernel<VB, ET>;
  const int64_t warps = (int64_t)((a.T + kCols - 1) / kCols) * a.E;
  launch(k, persistent_grid(k, kThreads, 0, (warps + kWarps - 1) / kWarps), kThreads, 0, s, a.x, a.x_stride, router,
         a.H, a.T, a.E, logits);
  return moe_topk_gating(logits, a.T, a.E, a.K, mode, normalize, top_expert, weights,
                         reinterpret_cast<moe_stream_t>(s));
}

template <int VB, typename ET> int run_rows(const LayerArgs& a, cudaStream_t s) {
  const size_t seg = segments_bytes(a.n, a.E);
  auto g = gate_up_rows_kernel<VB, ET>;
  launch(g, persistent_grid(g, kThreads, seg, ((a.n < a.E ? a.n : a.E) * a.F + kWarps - 1) / kWarps), kThreads, seg, s, a);
  const size_t down = seg + sizeof(float) * kWarps * a.T;
  auto d = down_rows_kernel<VB, ET>;
  launch(d, persistent_grid(d, kThreads, down, (a.H + kWarps - 1) / kWarps), kThreads, down, s, a);
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

template <int NT, int MT>
int launch_stream(const StreamArgs& p, const CUtensorMap& gate_up, const CUtensorMap& down, size_t seg, size_t ysum,
                  cudaStream_t s) {
  static std::atomic<int> granted_g[64], granted_d[64];
  auto g = gate_up_stream_kernel<NT>;
  auto d = down_stream_kernel<NT, MT>;
  const size_t ring = (size_t)kStages * p.stage_bytes + 1024;
  if (!allow_smem(g, (int)(ring + seg), granted_g) || !allow_smem(d, (int)(ring + seg + ysum), granted_d))
    return MOE_ERR_CUDA;
  const int64_t pairs = (p.a.n < p.a.E ? p.a.n : p.a.E) * p.a.F, sms = num_sms();
  launch(g, (unsigned)(pairs < sms ? pairs : sms), kStreamThreads, ring + seg, s, p, gate_up);
  launch(d, (unsigned)(p.a.H < sms ? p.a.H : sms), kStreamThreads, ring + seg + ysum, s, p, down);
  return check_launch();
}

template <int NT> int dispatch_stream(StreamArgs p, cudaStream_t s) {
  const int64_t sms = num_sms();
  const int64_t per_cta = (p.a.H + sms - 1) / sms;
  const int MT = per_cta <= 16 ? 1 : (per_cta <= 32 ? 2 : 4);
  p.down_rows = (int)(per_cta < 16 * MT ? per_cta : 16 * MT);
  const size_t seg = segments_bytes(p.a.n, p.a.E);
  const size_t ysum = sizeof(float) * p.a.T * p.down_rows;
  // Up to 16 tokens: stages such that a CTA of each kernel fits on an SM
  // together, so that the second kernel's first copies overlap the first's
  // end. Beyond: as large as fit, for the tokens' rows beside the weights'.
  p.stage_bytes = NT <= 2 ? 34816 : (int)((226304 - seg - ysum) / kStages / 1024 * 1024);
  if (p.stage_bytes > 65536) p.stage_bytes = 65536;
  p.gate_tokens = p.down_tokens = NT * 8;
  while (p.gate_tokens > 8 && stage_blocks(p.stage_bytes, 32, p.gate_tokens) < 1) p.gate_tokens -= 8;
  while (p.down_tokens > 8 && stage_blocks(p.stage_bytes, p.down_rows, 2 * p.down_tokens) < 1) p.down_tokens -= 8;
  CUtensorMap gate_up, down;
  if (!tensor_map(&gate_up, p.a.w_gate_up, p.a.H, p.a.F, 2 * (int64_t)p.a.E, 16, 2) ||
      !tensor_map(&down, p.a.w_down, p.a.F, p.a.H, p.a.E, p.down_rows, 1))
    return MOE_ERR_CUDA;
  switch (MT) {
    case 1: return launch_stream<NT, 1>(p, gate_up, down, seg, ysum, s);
    case 2: return launch_stream<NT, 2>(p, gate_up, down, seg, ysum, s);
    default: return launch_stream<NT, 4>(p, gate_up, down, seg, ysum, s);
  }
}

int run_stream(const LayerArgs& a, cudaStream_t s) {
  __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(a.h);
  const StreamArgs p{a, h, h + (int64_t)a.n * a.F, 0, 0, 0, 0};
  if (a.T <= 8) return dispatch_stream<1>(p, s);
  if (a.T <= 16) return dispatch_stream<2>(p, s);
  if (a.T <= 32) return dispatch_stream<4>(p, s);
  return dispatch_stream<8>(p, s);
}

template <typename ET>
int dispatch(const LayerArgs& a, const void* router, float* logits, int32_t mode, int32_t normalize,
             int32_t* top_expert, float* weights, cudaStream_t s) {
  constexpr int kE = 16 / Elem<ET>::kBytes;
  const bool by16 = a.H % kE == 0 && a.F % kE == 0 && a.x_stride % kE == 0 && aligned(a.x, 16) &&
                    aligned(a.w_gate_up, 16) && aligned(a.w_down, 16) && aligned(router, 16);
  const int rc = by16 ? run_router<16, ET>(a, router, logits, mode, normalize, top_expert, weights, s)
                      : run_router<Elem<ET>::kBytes, ET>(a, router, logits, mode, normalize, top_expert, weights, s);
  if (rc != MOE_OK) return rc;
  if (!by16) return run_rows<Elem<ET>::kBytes, ET>(a, s);
  if constexpr (Elem<ET>::kBytes == 2) {
    if (a.H >= kBlock && a.F >= kBlock) return run_stream(a, s);  // at least one box each way
  }
  return run_rows<16, ET>(a, s);
}

// Bytes of the workspace's parts: the logits, then h.
size_t logits_bytes(int64_t T, int32_t E) { return ((size_t)T * E * sizeof(float) + 255) / 256 * 256; }

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
  float* logits = static_cast<float*>(workspace);
  float* h = reinterpret_cast<float*>(static_cast<char*>(workspace) + logits_bytes(T, E));
  const LayerArgs a{x, w_gate_up, w_down, top_expert, weights, h, y, T > 1 ? x_stride : H, H, F,
                    (int32_t)T, E, K, (int32_t)(T * K), d_status};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MOE_F32) return dispatch<float>(a, router, logits, mode, normalize, top_out, weights_out, s);
  return dispatch<__nv_bfloat16>(a, router, logits, mode, normalize, top_out, weights_out, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_layer_workspace_size(int64_t T, int64_t H, int64_t F, int32_t E, int32_t K) {
  if (!sizes_ok(T, H, F, E, K) || !few(T, E, K)) return 0;
  return logits_bytes(T, E) + ((size_t)T * K * (size_t)F * sizeof(float) + 255) / 256 * 256 + 256;
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
