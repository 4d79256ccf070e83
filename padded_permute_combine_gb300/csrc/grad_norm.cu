// Global norm of many gradients, and clipping by it:
//   norm = sqrt(sum g^2),  out = g * min(1, max_norm / (norm + 1e-6)).
//
// The tensors are cut, on the host and once, into pieces of at most 32 KB; a
// kernel's CTAs stride over the pieces, so one launch covers any number of
// tensors of any sizes. Two launches: partial sums of squares, one per CTA,
// then either the norm (one CTA) or the scaling pass, whose CTAs each add the
// few hundred partial sums themselves. Bound by HBM: the norm reads each
// gradient once, clipping reads it twice (the coefficient depends on all of
// them) and writes it once. The scaling pass walks the pieces backwards, so
// the pieces that the first pass read last come from L2.
//
// Squares are added in fp32 within a thread's share of a piece (at most 64
// values) and in fp64 from there on; the order is fixed by the grid. A share
// whose fp32 sum overflows, is NaN, or falls below 2^-90 with a nonzero value
// in it is read and added again in fp64, so the norm is right over the whole
// range of the types.
#include <math.h>

#include "common.cuh"
#include "moe_block.h"

namespace moe {
namespace {

// 128 bytes of a piece a thread. 5.6 GB of fp32 clipped in 2.42 ms, 1.6 GB of
// bf16 summed in 233 us; with 512 threads, 64 KB and 4 CTAs 2.49 ms and 259 us,
// with 64 KB and 256 threads 2.50 ms and 298 us. More CTAs than fit at once
// (two or three) even out pieces of different lengths.
constexpr int kThreads = 256;
constexpr int64_t kPieceBytes = 32768;
constexpr int kCtasPerSm = 8;
constexpr int kMaxCtas = 2048;  // a partial sum each

// Plain (not read-only-path) loads: the scaling pass may write in place.
__device__ __forceinline__ u32x8 ld_vec(const u32x8* p) {
  u32x8 v;
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                 "=r"(v.w[7])
               : "l"(p)
               : "memory");
  return v;
}

template <typename ET> __device__ __forceinline__ float to_f32(ET v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename ET> __device__ __forceinline__ ET from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Elements before the first 32-byte boundary at or after p (at most n).
template <typename ET> __device__ __forceinline__ int head_elems(const void* p, int n) {
  const int h = (int)((32 - (reinterpret_cast<uintptr_t>(p) & 31)) & 31) / (int)sizeof(ET);
  return h < n ? h : n;
}

// Sum of squares of this thread's share of a piece, in fp32 or fp64.
template <typename ET, typename ACC>
__device__ __forceinline__ ACC share_sumsq(const ET* __restrict__ g, int n, uint32_t* nonzero) {
  constexpr int kE = 32 / (int)sizeof(ET);
  const int head = head_elems<ET>(g, n);
  const int vecs = (n - head) / kE;
  const int tail0 = head + vecs * kE;
  ACC s = 0;
  uint32_t nz = 0;
  auto add = [&](float v) {
    nz |= __float_as_uint(v) << 1;
    s += (ACC)v * (ACC)v;
  };
  if (threadIdx.x < head) add(to_f32<ET>(g[threadIdx.x]));
  if (tail0 + (int)threadIdx.x < n) add(to_f32<ET>(g[tail0 + threadIdx.x]));
  const u32x8* v = reinterpret_cast<const u32x8*>(g + head);
  constexpr int kU = (int)(kPieceBytes / 32 / kThreads);  // vectors per thread of a full piece
  u32x8 r[kU];
#pragma unroll
  for (int j = 0; j < kU; ++j) {
    const int i = (int)threadIdx.x + j * kThreads;
    r[j] = i < vecs ? ld_vec(v + i) : zero_vec<u32x8>();
  }
#pragma unroll
  for (int j = 0; j < kU; ++j) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      add(Elem<ET>::get(r[j].w[q], 0));
      if (sizeof(ET) == 2) add(Elem<ET>::get(r[j].w[q], 1));
    }
  }
  *nonzero = nz;
  return s;
}

template <typename ET> __device__ __forceinline__ double piece_sumsq(const void* grad, int n) {
  const ET* g = static_cast<const ET*>(grad);
  uint32_t nz;
  const float s = share_sumsq<ET, float>(g, n, &nz);
  // NaN fails both comparisons.
  if ((s >= 0x1p-90f && s <= 3.0e38f) || nz == 0) return (double)s;
  return share_sumsq<ET, double>(g, n, &nz);
}

// Sum over the CTA, in every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double s) {
  __shared__ double part[kThreads / kWarp];
#pragma unroll
  for (int d = kWarp / 2; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane_id() == 0) part[threadIdx.x / kWarp] = s;
  __syncthreads();
  double t = 0;
#pragma unroll
  for (int w = 0; w < kThreads / kWarp; ++w) t += part[w];
  return t;
}

__global__ void __launch_bounds__(kThreads)
    sumsq_kernel(const moe_grad_piece* __restrict__ pieces, int64_t P, double* __restrict__ partial) {
  await_previous_kernel();
  double s = 0;
  for (int64_t i = blockIdx.x; i < P; i += gridDim.x) {
    const moe_grad_piece p = pieces[i];
    s += p.dtype == MOE_F32 ? piece_sumsq<float>(p.grad, (int)p.numel)
                            : piece_sumsq<__nv_bfloat16>(p.grad, (int)p.numel);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__device__ __forceinline__ float total_norm(const double* partial, int parts) {
  double s = 0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += partial[i];
  return (float)sqrt(block_sum(s));
}

__global__ void __launch_bounds__(kThreads)
    norm_kernel(const double* __restrict__ partial, int parts, float* __restrict__ norm) {
  await_previous_kernel();
  const float n = total_norm(partial, parts);
  if (threadIdx.x == 0) *norm = n;
}

// A gradient and an output that lie differently to 32 bytes have no vectors in
// common and go element by element: 2^28 fp32 values 1.41 ms (0.48 where they
// lie alike), bf16 1.28 (0.25). The outs that a training program keeps are laid
// out like the gradients, or are the gradients.
template <typename ET> __device__ __forceinline__ void scale_piece(const void* grad, void* out, int n, float c) {
  constexpr int kE = 32 / (int)sizeof(ET);
  const ET* g = static_cast<const ET*>(grad);
  ET* o = static_cast<ET*>(out);
  if ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(o)) & 31) {
    for (int i = threadIdx.x; i < n; i += kThreads) o[i] = from_f32<ET>(to_f32<ET>(g[i]) * c);
    return;
  }
  const int head = head_elems<ET>(g, n);
  const int vecs = (n - head) / kE;
  const int tail0 = head + vecs * kE;
  if (threadIdx.x < head) o[threadIdx.x] = from_f32<ET>(to_f32<ET>(g[threadIdx.x]) * c);
  if (tail0 + (int)threadIdx.x < n) o[tail0 + threadIdx.x] = from_f32<ET>(to_f32<ET>(g[tail0 + threadIdx.x]) * c);
  const u32x8* v = reinterpret_cast<const u32x8*>(g + head);
  u32x8* w = reinterpret_cast<u32x8*>(o + head);
  constexpr int kU = (int)(kPieceBytes / 32 / kThreads);
  u32x8 r[kU];
#pragma unroll
  for (int j = 0; j < kU; ++j) {
    const int i = (int)threadIdx.x + j * kThreads;
    if (i < vecs) r[j] = ld_vec(v + i);
  }
#pragma unroll
  for (int j = 0; j < kU; ++j) {
    const int i = (int)threadIdx.x + j * kThreads;
    if (i >= vecs) break;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if constexpr (sizeof(ET) == 4) {
        r[j].w[q] = __float_as_uint(__uint_as_float(r[j].w[q]) * c);
      } else {
        r[j].w[q] = pack_bf16x2(Elem<ET>::get(r[j].w[q], 0) * c, Elem<ET>::get(r[j].w[q], 1) * c);
      }
    }
    st_stream(w + i, r[j]);
  }
}

__global__ void __launch_bounds__(kThreads)
    clip_kernel(const moe_grad_piece* __restrict__ pieces, int64_t P, const double* __restrict__ partial, int parts,
                float max_norm, float* __restrict__ norm) {
  await_previous_kernel();
  const float n = total_norm(partial, parts);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  float c = max_norm / (n + 1e-6f);
  if (c > 1.0f) c = 1.0f;  // NaN stays
  for (int64_t i = P - 1 - blockIdx.x; i >= 0; i -= gridDim.x) {
    const moe_grad_piece p = pieces[i];
    if (p.out == nullptr || (c == 1.0f && p.out == p.grad)) continue;
    if (p.dtype == MOE_F32)
      scale_piece<float>(p.grad, p.out, (int)p.numel, c);
    else
      scale_piece<__nv_bfloat16>(p.grad, p.out, (int)p.numel, c);
  }
}

// Cuts one tensor into pieces that end on 32-byte boundaries of the gradient; f(first element, elements).
template <typename F> void cut(const moe_grad_tensor& t, F f) {
  const int eb = dtype_bytes(t.dtype);
  const int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(t.grad) & 31) / eb;
  int64_t at = 0;
  while (at < t.numel) {
    int64_t m = kPieceBytes / eb - (at == 0 ? off : 0);
    if (m > t.numel - at) m = t.numel - at;
    f(at, m);
    at += m;
  }
}

bool valid(const moe_grad_tensor& t) {
  const int eb = dtype_bytes(t.dtype);
  if (eb == 0 || t.numel < 0 || (t.numel > 0 && t.grad == nullptr)) return false;
  return aligned(t.grad, eb) && aligned(t.out, eb);
}

int grid_of(int64_t P) {
  int64_t g = (int64_t)num_sms() * kCtasPerSm;
  if (g > kMaxCtas) g = kMaxCtas;
  return (int)(P < g ? (P < 1 ? 1 : P) : g);
}

int checks(const moe_grad_piece* pieces, int64_t P, const float* norm, const void* ws, size_t bytes) {
  if (P < 0 || (P > 0 && pieces == nullptr) || norm == nullptr || ws == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(pieces, 16) || !aligned(norm, 4) || !aligned(ws, 8)) return MOE_ERR_UNSUPPORTED;
  return bytes < moe_grad_norm_workspace_size() ? MOE_ERR_INVALID_ARG : MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int64_t moe_grad_table_pieces(const moe_grad_tensor* tensors, int64_t n) {
  if (n < 0 || (n > 0 && tensors == nullptr)) return -1;
  int64_t count = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (!valid(tensors[i])) return -1;
    cut(tensors[i], [&](int64_t, int64_t) { ++count; });
  }
  return count;
}

extern "C" int moe_grad_table_fill(const moe_grad_tensor* tensors, int64_t n, moe_grad_piece* pieces, int64_t P) {
  const int64_t count = moe_grad_table_pieces(tensors, n);
  if (count < 0 || P != count || (P > 0 && pieces == nullptr)) return MOE_ERR_INVALID_ARG;
  int64_t at = 0;
  for (int64_t i = 0; i < n; ++i) {
    const moe_grad_tensor& t = tensors[i];
    const int eb = dtype_bytes(t.dtype);
    cut(t, [&](int64_t first, int64_t m) {
      pieces[at++] = {static_cast<const char*>(t.grad) + first * eb,
                      t.out == nullptr ? nullptr : static_cast<char*>(t.out) + first * eb, m, t.dtype, 0};
    });
  }
  return MOE_OK;
}

extern "C" size_t moe_grad_norm_workspace_size(void) { return kMaxCtas * sizeof(double); }

extern "C" int moe_grad_norm(const moe_grad_piece* pieces, int64_t P, float* norm, void* workspace, size_t bytes,
                             moe_stream_t stream) {
  const int rc = checks(pieces, P, norm, workspace, bytes);
  if (rc != MOE_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  const int grid = grid_of(P);
  launch(sumsq_kernel, grid, kThreads, 0, s, pieces, P, partial);
  launch(norm_kernel, 1, kThreads, 0, s, (const double*)partial, grid, norm);
  return check_launch();
}

extern "C" int moe_clip_grads(const moe_grad_piece* pieces, int64_t P, float max_norm, float* norm, void* workspace,
                              size_t bytes, moe_stream_t stream) {
  const int rc = checks(pieces, P, norm, workspace, bytes);
  if (rc != MOE_OK) return rc;
  if (!(max_norm >= 0.0f)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  const int grid = grid_of(P);
  launch(sumsq_kernel, grid, kThreads, 0, s, pieces, P, partial);
  launch(clip_kernel, grid, kThreads, 0, s, pieces, P, (const double*)partial, grid, max_norm, norm);
  return check_launch();
}
