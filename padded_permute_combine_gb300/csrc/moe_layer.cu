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
#include <math.h>

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
// order[i]: assignment at sorted place i; the active experts, and where each
// begins in order.
struct Segments {
  int32_t* order;   // [n]
  int32_t* expert;  // [min(n, E)]
  int32_t* begin;   // [min(n, E) + 1]
  int32_t active;
};

__host__ __device__ inline size_t segments_bytes(int32_t n, int32_t E) {
  const int m = n < E ? n : E;
  return sizeof(int32_t) * ((size_t)2 * n + E + 2 * m + 2);
}

// Called by the whole CTA; warp 0 does the work.
__device__ __forceinline__ Segments sort_choices(const int32_t* __restrict__ top_expert, int32_t n, int32_t E,
                                                 int32_t* status, int32_t* smem) {
  const int m = n < E ? n : E;
  Segments s;
  s.order = smem;
  int32_t* local = smem + n;   // rank of an assignment within its expert
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
      int e = i < n ? top_expert[i] : -1;
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
      const int e = top_expert[i];
      if (e >= 0 && e < E) s.order[count[e] + local[i]] = i;
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
  const Segments s = sort_choices(a.top_expert, a.n, a.E, a.status, smem);
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
        const int t = s.order[i0 + c < last ? i0 + c : last] / a.K;
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
  const Segments s = sort_choices(a.top_expert, a.n, a.E, a.status, smem);
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
          if (lane == 0 && i0 + c <= last) sum[s.order[i0 + c] / a.K] += v;
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

// ------------------------------------------------------------------ host

template <int VB, typename ET>
int run_rows(const LayerArgs& a, const void* router, float* logits, int32_t mode, int32_t normalize,
             int32_t* top_expert, float* weights, cudaStream_t s) {
  if (router != nullptr) {
    auto k = router_rows_kernel<VB, ET>;
    const int64_t warps = (int64_t)((a.T + kCols - 1) / kCols) * a.E;
    launch(k, persistent_grid(k, kThreads, 0, (warps + kWarps - 1) / kWarps), kThreads, 0, s, a.x, a.x_stride, router,
           a.H, a.T, a.E, logits);
    const int rc = moe_topk_gating(logits, a.T, a.E, a.K, mode, normalize, top_expert, weights,
                                   reinterpret_cast<moe_stream_t>(s));
    if (rc != MOE_OK) return rc;
  }
  const size_t seg = segments_bytes(a.n, a.E);
  auto g = gate_up_rows_kernel<VB, ET>;
  launch(g, persistent_grid(g, kThreads, seg, ((a.n < a.E ? a.n : a.E) * a.F + kWarps - 1) / kWarps), kThreads, seg, s, a);
  const size_t down = seg + sizeof(float) * kWarps * a.T;
  auto d = down_rows_kernel<VB, ET>;
  launch(d, persistent_grid(d, kThreads, down, (a.H + kWarps - 1) / kWarps), kThreads, down, s, a);
  return check_launch();
}

template <typename ET>
int dispatch(const LayerArgs& a, const void* router, float* logits, int32_t mode, int32_t normalize,
             int32_t* top_expert, float* weights, cudaStream_t s) {
  constexpr int kE = 16 / Elem<ET>::kBytes;
  const bool by16 = a.H % kE == 0 && a.F % kE == 0 && a.x_stride % kE == 0 && aligned(a.x, 16) &&
                    aligned(a.w_gate_up, 16) && aligned(a.w_down, 16) && aligned(router, 16);
  if (by16) return run_rows<16, ET>(a, router, logits, mode, normalize, top_expert, weights, s);
  return run_rows<Elem<ET>::kBytes, ET>(a, router, logits, mode, normalize, top_expert, weights, s);
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
