// Layer norm over the last dimension, forward and backward.
//   forward:  y = (x - mean) * rstd * weight + bias
//   backward: dx = rstd * (v - sum(v)/H - xhat * sum(v*xhat)/H), v = dy * weight,
//             dweight = sum_rows dy * xhat, dbias = sum_rows dy
//
// Bound by HBM: forward reads x and writes y, backward reads x and dy and
// writes dx. A row stays in the registers of the threads that loaded it (one
// warp for short rows, one CTA otherwise): each element is read once, the
// variance is taken from the centred values, and the next row is loaded
// before the current one is reduced. In the backward pass a thread owns the
// same columns in every row it meets, so the two sums over rows live in its
// registers; each CTA writes one row of partial sums, and a second launch adds
// those in a fixed order. Rows too long for the registers take kernels that
// read a row again for each pass over it.
#include <math.h>

#include "common.cuh"
#include "moe_block.h"
#include "vec_math.cuh"

namespace moe {
namespace {

struct FwdArgs {
  const void* x;
  const void* weight;
  const void* bias;
  void* y;
  float* mean;
  float* rstd;
  int64_t x_stride, rows, H;
  float eps;
};

struct BwdArgs {
  const void* dy;
  const void* x;
  const void* weight;
  const float* mean;
  const float* rstd;
  void* dx;
  float* partial;  // [2][CTAs][H]: dweight's partial sums, then dbias's; nullptr when neither is asked for
  int64_t dy_stride, x_stride, rows, H;
};

template <typename ET> __device__ __forceinline__ float load1(const void* p, int64_t i);
template <> __device__ __forceinline__ float load1<float>(const void* p, int64_t i) {
  return __ldg(static_cast<const float*>(p) + i);
}
template <> __device__ __forceinline__ float load1<__nv_bfloat16>(const void* p, int64_t i) {
  return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + i));
}
__device__ __forceinline__ void store1(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, int64_t i, float v) { p[i] = __float2bfloat16_rn(v); }

// kE consecutive weights from column c (c and the array are aligned to the
// vector that a row uses), or `otherwise` where the array is absent.
template <typename WT, int kE>
__device__ __forceinline__ void load_cols(const void* w, int64_t c, float otherwise, float* out) {
  if (w == nullptr) {
#pragma unroll
    for (int q = 0; q < kE; ++q) out[q] = otherwise;
    return;
  }
  constexpr int kBytes = kE * Elem<WT>::kBytes;
  constexpr int kPart = kBytes > 16 ? 16 : kBytes;
  using L = Lanes<kPart, WT>;
  using V = typename L::V;
#pragma unroll
  for (int p = 0; p < kBytes / kPart; ++p) {
    const V v = ld_l1(reinterpret_cast<const V*>(static_cast<const char*>(w) + c * Elem<WT>::kBytes) + p);
#pragma unroll
    for (int q = 0; q < L::kElems; ++q) out[p * L::kElems + q] = L::get(v, q);
  }
}

// Sums of N values over the threads that share a row: a warp, or the CTA
// (`buf` alternates between two halves of `red`, so one barrier suffices).
template <int N, bool WARP_ROW> __device__ __forceinline__ void row_sum(float (&s)[N], float* red, int& buf) {
#pragma unroll
  for (int d = kWarp / 2; d > 0; d >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
  }
  if constexpr (!WARP_ROW) {
    const int warps = (int)blockDim.x / kWarp, lane = lane_id();
    float* r = red + buf * (N * kWarp);
    buf ^= 1;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[i * kWarp + threadIdx.x / kWarp] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = lane < warps ? r[i * kWarp + lane] : 0.0f;
#pragma unroll
      for (int d = kWarp / 2; d > 0; d >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
    }
  }
}

template <int VB, typename ET, typename WT, int NV, bool WARP_ROW, int MAXT>
__global__ void __launch_bounds__(MAXT) fwd_kernel(FwdArgs a) {
  using L = Lanes<VB, ET>;
  using V = typename L::V;
  constexpr int kE = L::kElems;
  __shared__ float red[2 * kWarp];
  await_previous_kernel();
  const int tid = WARP_ROW ? lane_id() : (int)threadIdx.x;
  const int tpr = WARP_ROW ? kWarp : (int)blockDim.x;
  const int64_t step = WARP_ROW ? (int64_t)gridDim.x * (blockDim.x / kWarp) : gridDim.x;
  const int64_t first = WARP_ROW ? (int64_t)blockIdx.x * (blockDim.x / kWarp) + threadIdx.x / kWarp : blockIdx.x;
  const int vecs = (int)(a.H / kE);
  const float inv_h = 1.0f / (float)a.H;
  int buf = 0;
  V nxt[NV];
  auto load = [&](int64_t row) {
    const V* p = reinterpret_cast<const V*>(static_cast<const char*>(a.x) + row * a.x_stride * Elem<ET>::kBytes);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * tpr;
      if (i < vecs) nxt[j] = ld_stream(p + i);
    }
  };
  if (first < a.rows) load(first);
  for (int64_t row = first; row < a.rows; row += step) {
    float v[NV][kE];
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = tid + j * tpr < vecs;
#pragma unroll
      for (int q = 0; q < kE; ++q) {
        v[j][q] = in ? L::get(nxt[j], q) : 0.0f;
        s[0] += v[j][q];
      }
    }
    if (row + step < a.rows) load(row + step);
    row_sum<1, WARP_ROW>(s, red, buf);
    const float mean = s[0] * inv_h;
    s[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (tid + j * tpr < vecs) {
#pragma unroll
        for (int q = 0; q < kE; ++q) {
          v[j][q] -= mean;
          s[0] += v[j][q] * v[j][q];
        }
      }
    }
    row_sum<1, WARP_ROW>(s, red, buf);
    const float rstd = rsqrtf(s[0] * inv_h + a.eps);
    if (tid == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    V* out = reinterpret_cast<V*>(static_cast<char*>(a.y) + row * a.H * Elem<ET>::kBytes);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * tpr;
      if (i >= vecs) break;
      float w[kE], b[kE], o[kE];
      load_cols<WT, kE>(a.weight, (int64_t)i * kE, 1.0f, w);
      load_cols<WT, kE>(a.bias, (int64_t)i * kE, 0.0f, b);
#pragma unroll
      for (int q = 0; q < kE; ++q) {
        o[q] = fmaf(v[j][q] * rstd, w[q], b[q]);
      }
      st_stream(out + i, L::pack(o));
    }
  }
}

template <int VB, typename ET, typename WT, int NV, bool WARP_ROW, int MAXT>
__global__ void __launch_bounds__(MAXT) bwd_kernel(BwdArgs a) {
  using L = Lanes<VB, ET>;
  using V = typename L::V;
  constexpr int kE = L::kElems;
  __shared__ float red[4 * kWarp];
  await_previous_kernel();
  const int tid = WARP_ROW ? lane_id() : (int)threadIdx.x;
  const int tpr = WARP_ROW ? kWarp : (int)blockDim.x;
  const int64_t step = WARP_ROW ? (int64_t)gridDim.x * (blockDim.x / kWarp) : gridDim.x;
  const int64_t first = WARP_ROW ? (int64_t)blockIdx.x * (blockDim.x / kWarp) + threadIdx.x / kWarp : blockIdx.x;
  const int vecs = (int)(a.H / kE);
  const float inv_h = 1.0f / (float)a.H;
  int buf = 0;
  float aw[NV][kE], ab[NV][kE];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int q = 0; q < kE; ++q) aw[j][q] = ab[j][q] = 0.0f;
  }
  V nx[NV], nd[NV];
  float nmean = 0.0f, nrstd = 0.0f;
  auto load = [&](int64_t row) {
    const V* px = reinterpret_cast<const V*>(static_cast<const char*>(a.x) + row * a.x_stride * Elem<ET>::kBytes);
    const V* pd = reinterpret_cast<const V*>(static_cast<const char*>(a.dy) + row * a.dy_stride * Elem<ET>::kBytes);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * tpr;
      nx[j] = i < vecs ? ld_stream(px + i) : zero_vec<V>();
      nd[j] = i < vecs ? ld_stream(pd + i) : zero_vec<V>();
    }
    nmean = __ldg(a.mean + row);
    nrstd = __ldg(a.rstd + row);
  };
  if (first < a.rows) load(first);
  for (int64_t row = first; row < a.rows; row += step) {
    V cx[NV], cd[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      cx[j] = nx[j];
      cd[j] = nd[j];
    }
    const float mean = nmean, rstd = nrstd;
    if (row + step < a.rows) load(row + step);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * tpr;
      if (i >= vecs) break;
      float w[kE];
      load_cols<WT, kE>(a.weight, (int64_t)i * kE, 1.0f, w);
#pragma unroll
      for (int q = 0; q < kE; ++q) {
        const float dy = L::get(cd[j], q);
        const float xhat = (L::get(cx[j], q) - mean) * rstd;
        const float v = dy * w[q];
        s[0] += v;
        s[1] += v * xhat;
        aw[j][q] += dy * xhat;
        ab[j][q] += dy;
      }
    }
    row_sum<2, WARP_ROW>(s, red, buf);
    const float c0 = s[0] * inv_h, c1 = s[1] * inv_h;
    V* out = reinterpret_cast<V*>(static_cast<char*>(a.dx) + row * a.H * Elem<ET>::kBytes);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * tpr;
      if (i >= vecs) break;
      float w[kE], o[kE];
      load_cols<WT, kE>(a.weight, (int64_t)i * kE, 1.0f, w);
#pragma unroll
      for (int q = 0; q < kE; ++q) {
        const float dy = L::get(cd[j], q);
        const float xhat = (L::get(cx[j], q) - mean) * rstd;
        const float v = dy * w[q];
        o[q] = rstd * (v - c0 - xhat * c1);
      }
      st_stream(out + i, L::pack(o));
    }
  }
  if (a.partial == nullptr) return;
  float* pw = a.partial + (int64_t)blockIdx.x * a.H;
  float* pb = pw + (int64_t)gridDim.x * a.H;
  if constexpr (!WARP_ROW) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = tid + j * tpr;
      if (i >= vecs) break;
#pragma unroll
      for (int q = 0; q < kE; ++q) {
        pw[(int64_t)i * kE + q] = aw[j][q];
        pb[(int64_t)i * kE + q] = ab[j][q];
      }
    }
  } else {
    // The CTA's warps hold the same columns: added warp by warp.
    extern __shared__ float acc[];  // [2][NV * 32 * kE]
    constexpr int kCols = NV * kWarp * kE;
    for (int w = 0; w < (int)(blockDim.x / kWarp); ++w) {
      if ((int)(threadIdx.x / kWarp) == w) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
          for (int q = 0; q < kE; ++q) {
            const int c = (tid + j * kWarp) * kE + q;
            acc[c] = (w ? acc[c] : 0.0f) + aw[j][q];
            acc[kCols + c] = (w ? acc[kCols + c] : 0.0f) + ab[j][q];
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < (int)a.H; c += blockDim.x) {
      pw[c] = acc[c];
      pb[c] = acc[kCols + c];
    }
  }
}

// Rows of any length, one CTA each: a pass for the mean, one for the variance, one to write.
template <typename ET, typename WT> __global__ void __launch_bounds__(512) fwd_long_kernel(FwdArgs a) {
  __shared__ float red[2 * kWarp];
  await_previous_kernel();
  const float inv_h = 1.0f / (float)a.H;
  int buf = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const ET* x = static_cast<const ET*>(a.x) + row * a.x_stride;
    float s[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < a.H; c += blockDim.x) s[0] += load1<ET>(x, c);
    row_sum<1, false>(s, red, buf);
    const float mean = s[0] * inv_h;
    s[0] = 0.0f;
    for (int64_t c = threadIdx.x; c < a.H; c += blockDim.x) {
      const float d = load1<ET>(x, c) - mean;
      s[0] += d * d;
    }
    row_sum<1, false>(s, red, buf);
    const float rstd = rsqrtf(s[0] * inv_h + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    for (int64_t c = threadIdx.x; c < a.H; c += blockDim.x) {
      const float xhat = (load1<ET>(x, c) - mean) * rstd;
      store1(static_cast<ET*>(a.y), row * a.H + c,
             fmaf(xhat, a.weight != nullptr ? load1<WT>(a.weight, c) : 1.0f,
                  a.bias != nullptr ? load1<WT>(a.bias, c) : 0.0f));
    }
  }
}

template <typename ET, typename WT> __global__ void __launch_bounds__(512) bwd_long_kernel(BwdArgs a) {
  __shared__ float red[4 * kWarp];
  await_previous_kernel();
  const float inv_h = 1.0f / (float)a.H;
  int buf = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const ET* x = static_cast<const ET*>(a.x) + row * a.x_stride;
    const ET* dy = static_cast<const ET*>(a.dy) + row * a.dy_stride;
    const float mean = __ldg(a.mean + row), rstd = __ldg(a.rstd + row);
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < a.H; c += blockDim.x) {
      const float v = load1<ET>(dy, c) * (a.weight != nullptr ? load1<WT>(a.weight, c) : 1.0f);
      s[0] += v;
      s[1] += v * ((load1<ET>(x, c) - mean) * rstd);
    }
    row_sum<2, false>(s, red, buf);
    for (int64_t c = threadIdx.x; c < a.H; c += blockDim.x) {
      const float v = load1<ET>(dy, c) * (a.weight != nullptr ? load1<WT>(a.weight, c) : 1.0f);
      store1(static_cast<ET*>(a.dx), row * a.H + c,
             rstd * (v - s[0] * inv_h - (load1<ET>(x, c) - mean) * rstd * (s[1] * inv_h)));
    }
  }
}

// Partial column sums of long rows: CTA (c, g) owns 256 columns and every gridDim.y-th row from g on.
template <typename ET> __global__ void __launch_bounds__(256) bwd_long_cols_kernel(BwdArgs a) {
  await_previous_kernel();
  const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= a.H) return;
  float sw = 0.0f, sb = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float dy = load1<ET>(a.dy, row * a.dy_stride + c);
    sw += dy * ((load1<ET>(a.x, row * a.x_stride + c) - __ldg(a.mean + row)) * __ldg(a.rstd + row));
    sb += dy;
  }
  a.partial[blockIdx.y * a.H + c] = sw;
  a.partial[((int64_t)gridDim.y + blockIdx.y) * a.H + c] = sb;
}

// Adds the CTAs' partial sums: 32 columns per CTA, its 16 warps each a share
// of the parts. blockIdx.y: 0 dweight, 1 dbias.
template <typename WT>
__global__ void __launch_bounds__(512) cols_kernel(const float* __restrict__ partial, int parts, int64_t H,
                                                   WT* dweight, WT* dbias) {
  __shared__ float red[16][kWarp];
  await_previous_kernel();
  WT* out = blockIdx.y == 0 ? dweight : dbias;
  if (out == nullptr) return;
  const int lane = lane_id(), warp = threadIdx.x / kWarp;
  const int64_t c = (int64_t)blockIdx.x * kWarp + lane;
  float s = 0.0f;
  if (c < H) {
    const float* p = partial + (int64_t)blockIdx.y * parts * H + c;
#pragma unroll 4
    for (int g = warp; g < parts; g += 16) s += __ldcg(p + (int64_t)g * H);
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < H) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) t += red[w][lane];
    store1(out, c, t);
  }
}

// ------------------------------------------------------------------ host

constexpr int kRowWarps = 8;     // rows per CTA when a warp takes a row
constexpr int kMaxParts = 304;   // CTAs of the backward pass, each with a row of partial column sums

struct RowShape {
  bool warp_row;
  int nv, threads;  // threads == 0: the row does not fit
};

// Vectors per thread (a power of two up to max_nv) and threads per row.
RowShape row_shape(int64_t vecs, int max_nv, int want_threads, int max_threads) {
  if (vecs <= kWarp * 4) return {true, vecs <= kWarp ? 1 : (vecs <= kWarp * 2 ? 2 : 4), kRowWarps * kWarp};
  for (int limit : {want_threads, max_threads}) {
    for (int nv = 1; nv <= max_nv; nv <<= 1) {
      const int64_t t = ((vecs + nv - 1) / nv + kWarp - 1) / kWarp * kWarp;
      if (t <= limit) return {false, nv, (int)t};
    }
  }
  return {false, 0, 0};
}

int bwd_parts(int64_t rows) { return (int)(rows < kMaxParts ? rows : kMaxParts); }

template <int VB, typename ET, typename WT, int NV>
int launch_fwd(const FwdArgs& a, const RowShape& r, cudaStream_t s) {
  if (r.warp_row) {
    if constexpr (NV <= 4) {
      auto k = fwd_kernel<VB, ET, WT, NV, true, kRowWarps * kWarp>;
      launch(k, persistent_grid(k, r.threads, 0, (a.rows + kRowWarps - 1) / kRowWarps), r.threads, 0, s, a);
    }
  } else if (r.threads <= 256) {
    auto k = fwd_kernel<VB, ET, WT, NV, false, 256>;
    launch(k, persistent_grid(k, r.threads, 0, a.rows), r.threads, 0, s, a);
  } else {
    auto k = fwd_kernel<VB, ET, WT, NV, false, 1024>;
    launch(k, persistent_grid(k, r.threads, 0, a.rows), r.threads, 0, s, a);
  }
  return check_launch();
}

template <int VB, typename ET, typename WT> int dispatch_fwd(const FwdArgs& a, cudaStream_t s) {
  const RowShape r = row_shape(a.H / Lanes<VB, ET>::kElems, VB == 16 ? 4 : 16, 256, 1024);
  switch (r.nv) {
    case 1: return launch_fwd<VB, ET, WT, 1>(a, r, s);
    case 2: return launch_fwd<VB, ET, WT, 2>(a, r, s);
    case 4: return launch_fwd<VB, ET, WT, 4>(a, r, s);
    default: break;
  }
  if constexpr (VB != 16) {
    if (r.nv == 8) return launch_fwd<VB, ET, WT, 8>(a, r, s);
    if (r.nv == 16) return launch_fwd<VB, ET, WT, 16>(a, r, s);
  }
  auto k = fwd_long_kernel<ET, WT>;
  launch(k, persistent_grid(k, 512, 0, a.rows), 512, 0, s, a);
  return check_launch();
}

template <int VB, typename ET, typename WT, int NV>
int launch_bwd(const BwdArgs& a, const RowShape& r, int* parts, cudaStream_t s) {
  const int64_t most = bwd_parts(a.rows);
  auto go = [&](auto k, size_t smem, int64_t work) {
    const int grid = persistent_grid(k, r.threads, smem, work < most ? work : most);
    *parts = grid;
    launch(k, grid, r.threads, smem, s, a);
  };
  if (r.warp_row) {
    if constexpr (NV <= 4)
      go(bwd_kernel<VB, ET, WT, NV, true, kRowWarps * kWarp>, sizeof(float) * 2 * NV * kWarp * Lanes<VB, ET>::kElems,
         (a.rows + kRowWarps - 1) / kRowWarps);
  } else {
    go(bwd_kernel<VB, ET, WT, NV, false, 512>, 0, a.rows);
  }
  return check_launch();
}

template <int VB, typename ET, typename WT> int dispatch_bwd(const BwdArgs& a, int* parts, cudaStream_t s) {
  const RowShape r = row_shape(a.H / Lanes<VB, ET>::kElems, VB == 16 ? 4 : 16, 512, 512);
  switch (r.nv) {
    case 1: return launch_bwd<VB, ET, WT, 1>(a, r, parts, s);
    case 2: return launch_bwd<VB, ET, WT, 2>(a, r, parts, s);
    case 4: return launch_bwd<VB, ET, WT, 4>(a, r, parts, s);
    default: break;
  }
  if constexpr (VB != 16) {
    if (r.nv == 8) return launch_bwd<VB, ET, WT, 8>(a, r, parts, s);
    if (r.nv == 16) return launch_bwd<VB, ET, WT, 16>(a, r, parts, s);
  }
  auto k = bwd_long_kernel<ET, WT>;
  launch(k, persistent_grid(k, 512, 0, a.rows), 512, 0, s, a);
  *parts = bwd_parts(a.rows);
  if (a.partial != nullptr) {
    if (*parts > 32) *parts = 32;
    launch(bwd_long_cols_kernel<ET>, dim3((unsigned)((a.H + 255) / 256), (unsigned)*parts), 256, 0, s, a);
  }
  return check_launch();
}

// Rows are read and written in 16-byte vectors when their lengths, strides
// and addresses allow, else element by element.
template <typename ET> bool rows_by_16(int64_t H, const int64_t* strides, int ns, const void* const* ptrs, int np) {
  bool ok = H % (16 / Elem<ET>::kBytes) == 0;
  for (int i = 0; i < ns; ++i) ok = ok && strides[i] % (16 / Elem<ET>::kBytes) == 0;
  for (int i = 0; i < np; ++i) ok = ok && aligned(ptrs[i], 16);
  return ok;
}

int shape_checks(int32_t dtype, int32_t wdtype, int64_t rows, int64_t H) {
  if (rows < 0 || H < 1) return MOE_ERR_INVALID_ARG;
  if (dtype_bytes(dtype) == 0 || dtype_bytes(wdtype) == 0) return MOE_ERR_UNSUPPORTED;
  if (H > INT32_MAX / 2 || (rows > 0 && H > INT64_MAX / 8 / rows)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool bad_stride(int64_t stride, int64_t rows, int64_t H) {
  return rows > 1 && (stride < H || stride > INT64_MAX / 8 / rows);
}

template <typename ET, typename WT> int run_fwd(FwdArgs a, cudaStream_t s) {
  if (a.rows < 2) a.x_stride = a.H;
  const void* ptrs[] = {a.x, a.y, a.weight, a.bias};
  if (rows_by_16<ET>(a.H, &a.x_stride, 1, ptrs, 4)) return dispatch_fwd<16, ET, WT>(a, s);
  return dispatch_fwd<Elem<ET>::kBytes, ET, WT>(a, s);
}

template <typename ET, typename WT> int run_bwd(BwdArgs a, void* dweight, void* dbias, cudaStream_t s) {
  if (a.rows < 2) a.x_stride = a.dy_stride = a.H;
  int parts = 0, rc = MOE_OK;
  if (a.rows > 0) {
    const int64_t strides[] = {a.x_stride, a.dy_stride};
    const void* ptrs[] = {a.x, a.dy, a.dx, a.weight};
    rc = rows_by_16<ET>(a.H, strides, 2, ptrs, 4) ? dispatch_bwd<16, ET, WT>(a, &parts, s)
                                                  : dispatch_bwd<Elem<ET>::kBytes, ET, WT>(a, &parts, s);
  }
  if (rc != MOE_OK || (dweight == nullptr && dbias == nullptr)) return rc;
  launch(cols_kernel<WT>, dim3((unsigned)((a.H + kWarp - 1) / kWarp), 2), 512, 0, s, (const float*)a.partial, parts,
         a.H, static_cast<WT*>(dweight), static_cast<WT*>(dbias));
  return check_launch();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_layer_norm_fwd(const void* x, int32_t dtype, int64_t x_stride, const void* weight, const void* bias,
                                  int32_t wdtype, int64_t rows, int64_t H, float eps, void* y, float* mean,
                                  float* rstd, moe_stream_t stream) {
  const int rc = shape_checks(dtype, wdtype, rows, H);
  if (rc != MOE_OK) return rc;
  if (!(eps >= 0.0f) || bad_stride(x_stride, rows, H)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (x == nullptr || y == nullptr)) return MOE_ERR_INVALID_ARG;
  const int eb = dtype_bytes(dtype), wb = dtype_bytes(wdtype);
  if (!aligned(x, eb) || !aligned(y, eb) || !aligned(weight, wb) || !aligned(bias, wb) || !aligned(mean, 4) ||
      !aligned(rstd, 4))
    return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const FwdArgs a{x, weight, bias, y, mean, rstd, x_stride, rows, H, eps};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MOE_F32) return wdtype == MOE_F32 ? run_fwd<float, float>(a, s) : run_fwd<float, __nv_bfloat16>(a, s);
  return wdtype == MOE_F32 ? run_fwd<__nv_bfloat16, float>(a, s) : run_fwd<__nv_bfloat16, __nv_bfloat16>(a, s);
}

extern "C" size_t moe_layer_norm_bwd_workspace_size(int64_t rows, int64_t H) {
  if (rows < 0 || H < 1) return 0;
  return (size_t)bwd_parts(rows < 1 ? 1 : rows) * 2 * (size_t)H * sizeof(float);
}

extern "C" int moe_layer_norm_bwd(const void* dy, int64_t dy_stride, const void* x, int32_t dtype, int64_t x_stride,
                                  const void* weight, int32_t wdtype, const float* mean, const float* rstd,
                                  int64_t rows, int64_t H, void* dx, void* dweight, void* dbias, void* workspace,
                                  size_t workspace_bytes, moe_stream_t stream) {
  const int rc = shape_checks(dtype, wdtype, rows, H);
  if (rc != MOE_OK) return rc;
  if (bad_stride(x_stride, rows, H) || bad_stride(dy_stride, rows, H)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (dy == nullptr || x == nullptr || dx == nullptr || mean == nullptr || rstd == nullptr))
    return MOE_ERR_INVALID_ARG;
  const bool cols = dweight != nullptr || dbias != nullptr;
  if (cols && (workspace == nullptr || workspace_bytes < moe_layer_norm_bwd_workspace_size(rows, H)))
    return MOE_ERR_INVALID_ARG;
  const int eb = dtype_bytes(dtype), wb = dtype_bytes(wdtype);
  if (!aligned(dy, eb) || !aligned(x, eb) || !aligned(dx, eb) || !aligned(weight, wb) || !aligned(dweight, wb) ||
      !aligned(dbias, wb) || !aligned(mean, 4) || !aligned(rstd, 4) || (cols && !aligned(workspace, 16)))
    return MOE_ERR_UNSUPPORTED;
  if (rows == 0 && !cols) return MOE_OK;
  const BwdArgs a{dy, x, weight, mean, rstd, dx, cols ? static_cast<float*>(workspace) : nullptr,
                  dy_stride, x_stride, rows, H};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MOE_F32)
    return wdtype == MOE_F32 ? run_bwd<float, float>(a, dweight, dbias, s)
                             : run_bwd<float, __nv_bfloat16>(a, dweight, dbias, s);
  return wdtype == MOE_F32 ? run_bwd<__nv_bfloat16, float>(a, dweight, dbias, s)
                           : run_bwd<__nv_bfloat16, __nv_bfloat16>(a, dweight, dbias, s);
}
