// Layer norm over the last dimension, forward and backward.
//   forward:  y = (x - mean) * rstd * weight + bias
//   backward: dx = rstd * (v - sum(v)/H - xhat * sum(v*xhat)/H), v = dy * weight,
//             dweight = sum_rows dy * xhat, dbias = sum_rows dy
//
// Bound by HBM: forward reads x and writes y, backward reads x and dy and
// writes dx. A row stays in the registers of the threads that loaded it (8, 16
// or 32 lanes for short rows, a CTA otherwise): each element is read once and
// the variance is taken from the centred values. The next rows (DEPTH of them)
// are on their way into registers while one is reduced. In the backward pass a
// thread owns the same columns in every row it meets, so the two sums over
// rows live in its registers; each CTA writes one row of partial sums, and a
// second launch adds those in a fixed order. The backward pass takes rows of
// more than 512 bytes through a ring in shared memory: bf16 up to 32 KB, fp32 up
// to 16 KB and from 32 to 50 KB (between, they stay in registers). Packed rows
// that 16 bytes do not divide go through shared memory eight at a time. Rows
// too long for the registers take kernels that read a row again for each pass
// over it.
#include <math.h>

#include <atomic>

#include "block_common.h"
#include "bulk.cuh"
#include "common.cuh"
#include "moe_block.h"
#include "vec_math.cuh"

namespace moe {
namespace {

constexpr int kMaxThreads = 1024;  // of a CTA that takes a row
constexpr int kRowWarps = 8;       // warps of a CTA whose lanes share rows: up to 85 registers

struct FwdArgs {
  const void* x;
  const void* weight;
  const void* bias;
  void* y;
  float* mean;
  float* rstd;
  int64_t x_stride, rows, H;
  float eps;
  int waits;  // for rows' copies: 1, or 0 (all give up at once) in tests
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
  int waits;
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

// A row's values in registers: pairs for the packed fp32 instructions where a
// vector holds several elements (they halve the arithmetic, which bounded the
// bf16 kernels: 4.2 TB/s without them), single floats otherwise.
template <int kE> struct Pack {
  using T = uint64_t;
  static constexpr int N = kE / 2;
  __device__ __forceinline__ static T splat(float v) { return f2_pack(__float_as_uint(v), __float_as_uint(v)); }
  template <typename ET, typename V> __device__ __forceinline__ static T get(const V& v, int q) { return f2_elems<ET>(v, q); }
  __device__ __forceinline__ static T add(T a, T b) { return f2_add(a, b); }
  __device__ __forceinline__ static T sub(T a, T b) { return f2_sub(a, b); }
  __device__ __forceinline__ static T mul(T a, T b) { return f2_mul(a, b); }
  __device__ __forceinline__ static T fma(T a, T b, T c) { return f2_fma(a, b, c); }
  __device__ __forceinline__ static void put(T v, float* out) { f2_unpack(v, out[0], out[1]); }
  __device__ __forceinline__ static float sum(T v) {
    float a, b;
    f2_unpack(v, a, b);
    return a + b;
  }
};
template <> struct Pack<1> {
  using T = float;
  static constexpr int N = 1;
  __device__ __forceinline__ static T splat(float v) { return v; }
  template <typename ET, typename V> __device__ __forceinline__ static T get(const V& v, int) {
    return Lanes<Elem<ET>::kBytes, ET>::get(v, 0);
  }
  __device__ __forceinline__ static T add(T a, T b) { return a + b; }
  __device__ __forceinline__ static T sub(T a, T b) { return a - b; }
  __device__ __forceinline__ static T mul(T a, T b) { return __fmul_rn(a, b); }
  __device__ __forceinline__ static T fma(T a, T b, T c) { return fmaf(a, b, c); }
  __device__ __forceinline__ static void put(T v, float* out) { *out = v; }
  __device__ __forceinline__ static float sum(T v) { return v; }
};

// kE consecutive weights from column c (c and the array are aligned to the
// vector that a row uses), or `otherwise` where the array is absent.
template <typename WT, int kE>
__device__ __forceinline__ void load_cols(const void* w, int64_t c, float otherwise, typename Pack<kE>::T* out) {
  using P = Pack<kE>;
  if (w == nullptr) {
#pragma unroll
    for (int q = 0; q < P::N; ++q) out[q] = P::splat(otherwise);
    return;
  }
  // One load of up to 32 bytes: two of 16 would each touch every other half line.
  using V = typename Lanes<kE * Elem<WT>::kBytes, WT>::V;
  const V v = ld_l1(reinterpret_cast<const V*>(static_cast<const char*>(w) + c * Elem<WT>::kBytes));
#pragma unroll
  for (int q = 0; q < P::N; ++q) out[q] = P::template get<WT>(v, q);
}

// Sums of N values over LPR lanes, in each of them.
template <int N, int LPR> __device__ __forceinline__ void lane_sum(float (&s)[N]) {
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
  }
}

// Sums of N values over the threads that share a row: LPR lanes of a warp, or
// (LPR 0) the CTA, where `buf` alternates between two halves of `red`, so that
// one barrier suffices.
template <int N, int LPR> __device__ __forceinline__ void row_sum(float (&s)[N], float* red, int& buf) {
  lane_sum<N, LPR ? LPR : kWarp>(s);
  if constexpr (LPR == 0) {
    const int warps = (int)blockDim.x / kWarp, lane = lane_id();
    float* r = red + buf * (N * kWarp);
    buf ^= 1;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[i * kWarp + threadIdx.x / kWarp] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = lane < warps ? r[i * kWarp + lane] : 0.0f;
    lane_sum<N, kWarp>(s);
  }
}

// The rows that a thread works on: rows0 + i * step for its group of LPR lanes
// (or its CTA). Warps stay together: a group past the last row idles.
template <int LPR> struct Rows {
  int tid, tpr;
  int64_t at, step, warp_at;
  __device__ Rows() {
    if constexpr (LPR == 0) {
      tid = threadIdx.x;
      tpr = blockDim.x;
      at = warp_at = blockIdx.x;
      step = gridDim.x;
    } else {
      constexpr int kPer = kWarp / LPR;
      tid = threadIdx.x % LPR;
      tpr = LPR;
      warp_at = ((int64_t)blockIdx.x * (blockDim.x / kWarp) + threadIdx.x / kWarp) * kPer;
      at = warp_at + lane_id() / LPR;
      step = (int64_t)gridDim.x * (blockDim.x / kWarp) * kPer;
    }
  }
};

// FULL: every thread of the CTA has all its vectors and needs no masks; three
// CTAs an SM then, 80 registers a thread (8192 x 7168 bf16: 43 us, with masks 45;
// at 134 registers and two CTAs 62).
template <int VB, typename ET, typename WT, int NV, int LPR, int DEPTH, int MAXT, bool FULL>
__global__ void __launch_bounds__(LPR ? kRowWarps * kWarp : MAXT, LPR || (FULL && MAXT == 256) ? 3 : 1) fwd_kernel(FwdArgs a) {
  using L = Lanes<VB, ET>;
  using V = typename L::V;
  constexpr int kE = L::kElems;
  __shared__ float red[2 * 3 * kWarp];
  await_previous_kernel();
  const Rows<LPR> r;
  const int vecs = (int)(a.H / kE);
  const float inv_h = 1.0f / (float)a.H;
  int buf = 0;
  using P = Pack<kE>;
  using T = typename P::T;
  // Elements of the row in this warp (or group), and one over it.
  int held = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int left = vecs - (LPR ? 0 : (int)(threadIdx.x / kWarp) * kWarp) - j * r.tpr;
    held += left < 0 ? 0 : (left < (LPR ? LPR : kWarp) ? left : (LPR ? LPR : kWarp));
  }
  const float n_warp = (float)(held * kE), inv_warp = held ? 1.0f / n_warp : 0.0f;
  V ahead[DEPTH][NV];
  auto load = [&](V (&v)[NV], int64_t row) {
    if (FULL && row >= a.rows) row = a.rows - 1;  // read again and left; a branch here keeps the load from running ahead
    const V* p = reinterpret_cast<const V*>(static_cast<const char*>(a.x) + row * a.x_stride * Elem<ET>::kBytes);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = r.tid + j * r.tpr;
      v[j] = FULL || (i < vecs && row < a.rows) ? ld_stream(p + i) : zero_vec<V>();
    }
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(ahead[d], r.at + d * r.step);
  for (int64_t done = 0; r.warp_at + done < a.rows;) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int64_t row = r.at + done;
      if (r.warp_at + done >= a.rows) break;
      done += r.step;
      T v[NV][P::N], t = P::splat(0.0f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int q = 0; q < P::N; ++q) {
          v[j][q] = P::template get<ET>(ahead[d][j], q);
          t = P::add(t, v[j][q]);
        }
      }
      load(ahead[d], row + DEPTH * r.step);
      // Mean and squared deviations of the warp's part, then those of the row:
      // sum (x - mean)^2 = sum over warps of (sum (x - m_w)^2 + n_w (m_w - mean)^2).
      float s[1] = {P::sum(t)};
      lane_sum<1, LPR ? LPR : kWarp>(s);
      float mean = s[0] * inv_warp;
      const T part = P::splat(mean);
      t = P::splat(0.0f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!FULL && r.tid + j * r.tpr >= vecs) break;
#pragma unroll
        for (int q = 0; q < P::N; ++q) {
          const T c = P::sub(v[j][q], part);
          t = P::fma(c, c, t);
        }
      }
      float dev[1] = {P::sum(t)};
      lane_sum<1, LPR ? LPR : kWarp>(dev);
      if constexpr (LPR == 0) {
        const int warps = (int)blockDim.x / kWarp, lane = lane_id();
        float* b = red + buf * (3 * kWarp);
        buf ^= 1;
        if (lane == 0) {
          b[threadIdx.x / kWarp] = s[0];
          b[kWarp + threadIdx.x / kWarp] = dev[0];
          b[2 * kWarp + threadIdx.x / kWarp] = n_warp;
        }
        __syncthreads();
        const bool in = lane < warps;
        const float ws = in ? b[lane] : 0.0f, wd = in ? b[kWarp + lane] : 0.0f, wn = in ? b[2 * kWarp + lane] : 0.0f;
        s[0] = ws;
        lane_sum<1, kWarp>(s);
        mean = s[0] * inv_h;
        const float off = wn > 0.0f ? ws / wn - mean : 0.0f;
        dev[0] = fmaf(wn * off, off, wd);
        lane_sum<1, kWarp>(dev);
      }
      const float rstd = rsqrtf(dev[0] * inv_h + a.eps);
      if (!FULL && row >= a.rows) continue;
      if (r.tid == 0) {
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
      }
      V* out = reinterpret_cast<V*>(static_cast<char*>(a.y) + row * a.H * Elem<ET>::kBytes);
      const T m2 = P::splat(mean), r2 = P::splat(rstd);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = r.tid + j * r.tpr;
        if (!FULL && i >= vecs) break;
        T w[P::N], b[P::N];
        float o[kE];
        load_cols<WT, kE>(a.weight, (int64_t)i * kE, 1.0f, w);
        load_cols<WT, kE>(a.bias, (int64_t)i * kE, 0.0f, b);
#pragma unroll
        for (int q = 0; q < P::N; ++q) P::put(P::fma(P::mul(P::sub(v[j][q], m2), r2), w[q], b[q]), o + q * (kE / P::N));
        st_stream(out + i, L::pack(o));
      }
    }
  }
}

template <int VB, typename ET, typename WT, int NV, int LPR, int DEPTH, int MAXT>
__global__ void __launch_bounds__(LPR ? kRowWarps * kWarp : MAXT, LPR ? 3 : 1) bwd_kernel(BwdArgs a) {
  using L = Lanes<VB, ET>;
  using V = typename L::V;
  constexpr int kE = L::kElems;
  __shared__ float red[4 * kWarp];
  await_previous_kernel();
  const Rows<LPR> r;
  const int vecs = (int)(a.H / kE);
  const float inv_h = 1.0f / (float)a.H;
  int buf = 0;
  using P = Pack<kE>;
  using T = typename P::T;
  T aw2[NV][P::N], ab2[NV][P::N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int q = 0; q < P::N; ++q) aw2[j][q] = ab2[j][q] = P::splat(0.0f);
  }
  T w[NV][P::N];  // this thread's columns in every row
#pragma unroll
  for (int j = 0; j < NV; ++j)
    load_cols<WT, kE>(r.tid + j * r.tpr < vecs ? a.weight : nullptr, (int64_t)(r.tid + j * r.tpr) * kE, 1.0f, w[j]);
  V nx[DEPTH][NV], nd[DEPTH][NV];
  float nmean[DEPTH], nrstd[DEPTH];
  auto load = [&](int d, int64_t row) {
    const V* px = reinterpret_cast<const V*>(static_cast<const char*>(a.x) + row * a.x_stride * Elem<ET>::kBytes);
    const V* pd = reinterpret_cast<const V*>(static_cast<const char*>(a.dy) + row * a.dy_stride * Elem<ET>::kBytes);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = r.tid + j * r.tpr;
      const bool in = i < vecs && row < a.rows;
      nx[d][j] = in ? ld_stream(px + i) : zero_vec<V>();
      nd[d][j] = in ? ld_stream(pd + i) : zero_vec<V>();
    }
    nmean[d] = row < a.rows ? __ldg(a.mean + row) : 0.0f;
    nrstd[d] = row < a.rows ? __ldg(a.rstd + row) : 0.0f;
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(d, r.at + d * r.step);
  for (int64_t done = 0; r.warp_at + done < a.rows;) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int64_t row = r.at + done;
      if (r.warp_at + done >= a.rows) break;
      done += r.step;
      T xhat[NV][P::N], v[NV][P::N], s0 = P::splat(0.0f), s1 = s0;
      const T r2 = P::splat(nrstd[d]), m2 = P::splat(nmean[d]);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = r.tid + j * r.tpr;
        if (i >= vecs) break;
#pragma unroll
        for (int q = 0; q < P::N; ++q) {
          const T dy = P::template get<ET>(nd[d][j], q);
          xhat[j][q] = P::mul(P::sub(P::template get<ET>(nx[d][j], q), m2), r2);
          v[j][q] = P::mul(dy, w[j][q]);
          s0 = P::add(s0, v[j][q]);
          s1 = P::fma(v[j][q], xhat[j][q], s1);
          aw2[j][q] = P::fma(dy, xhat[j][q], aw2[j][q]);  // a row past the last has dy = 0
          ab2[j][q] = P::add(ab2[j][q], dy);
        }
      }
      load(d, row + DEPTH * r.step);
      float s[2] = {P::sum(s0), P::sum(s1)};
      row_sum<2, LPR>(s, red, buf);
      if (row >= a.rows) continue;
      const T c0 = P::splat(s[0] * inv_h), c1 = P::splat(-s[1] * inv_h);
      V* out = reinterpret_cast<V*>(static_cast<char*>(a.dx) + row * a.H * Elem<ET>::kBytes);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = r.tid + j * r.tpr;
        if (i >= vecs) break;
        float o[kE];
#pragma unroll
        for (int q = 0; q < P::N; ++q)
          P::put(P::mul(P::fma(xhat[j][q], c1, P::sub(v[j][q], c0)), r2), o + q * (kE / P::N));
        st_stream(out + i, L::pack(o));
      }
    }
  }
  if (a.partial == nullptr) return;
  float aw[NV][kE], ab[NV][kE];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int q = 0; q < P::N; ++q) {
      P::put(aw2[j][q], &aw[j][q * (kE / P::N)]);
      P::put(ab2[j][q], &ab[j][q * (kE / P::N)]);
    }
  }
  float* pw = a.partial + (int64_t)blockIdx.x * a.H;
  float* pb = pw + (int64_t)gridDim.x * a.H;
  if constexpr (LPR == 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = r.tid + j * r.tpr;
      if (i >= vecs) break;
#pragma unroll
      for (int q = 0; q < kE; ++q) {
        pw[(int64_t)i * kE + q] = aw[j][q];
        pb[(int64_t)i * kE + q] = ab[j][q];
      }
    }
  } else {
    // The CTA's groups hold the same columns: added within a warp, then warp by warp.
    extern __shared__ float acc[];  // [2][NV * LPR * kE]
    constexpr int kCols = NV * LPR * kE;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int q = 0; q < kE; ++q) {
#pragma unroll
        for (int d = LPR; d < kWarp; d <<= 1) {
          aw[j][q] += __shfl_xor_sync(0xffffffffu, aw[j][q], d);
          ab[j][q] += __shfl_xor_sync(0xffffffffu, ab[j][q], d);
        }
      }
    }
    for (int w = 0; w < (int)(blockDim.x / kWarp); ++w) {
      if ((int)(threadIdx.x / kWarp) == w && lane_id() < LPR) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
          for (int q = 0; q < kE; ++q) {
            const int c = (r.tid + j * LPR) * kE + q;
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

constexpr float kNaN = __builtin_nanf("");

// ------------------------------------------- rows through shared memory
//
// The backward pass for rows of more than 512 bytes. Up to 16 KB: two 16-byte
// vectors of the row per thread, two consecutive rows at a time. Above, up to 32
// KB of bf16 and from 32 to 50 of fp32, where a second reading of the rows would
// follow (2000 x 9000 fp32 56 us instead of 111, 4000 x 12800 99 instead of
// 259): four vectors and one row; fp32 rows of 16 to 32 KB fit in registers and
// take bwd_kernel. The rows are copied into a ring of slots
// by bulk copies (one for both rows where they are adjacent). What that buys
// over loads into registers: the copies ahead cost none (they read x and dy
// from the slot again after the sums instead of keeping them), and one barrier
// and one round of exchanges serve two rows. Those are a warp's cost whatever
// it holds: with one vector a thread they bounded the kernel (79 instead of 73
// us at 8192 x 7168 bf16, 84 with loads into registers). A slot is free again
// after the next iteration's barrier. Waits are bounded. A thread that gave up
// makes the CTA's rows NaN from then on, and its columns; the one that copies
// also waits once more (bounded) for what is on its way, and copies no more.
// (The forward pass gains nothing this way: 47 us instead of 43.)

constexpr int kRingThreads = 512;
// fp32 with four vectors a thread: up to 31 warps (one place of the sums is no warp's), for rows of 32 to 50 KB.
// Registers and shared memory decide how many CTAs an SM holds.
template <typename ET> __host__ __device__ constexpr int ring_registers(int nv) { return nv == 2 ? 96 : Elem<ET>::kBytes == 4 ? 64 : 128; }
template <typename ET> constexpr int ring_threads(int nv) { return nv == 4 && Elem<ET>::kBytes == 4 ? (kWarp - 1) * kWarp : kRingThreads; }
constexpr int kMaxSlots = 16;
constexpr int kRingSm = 200 * 1024;  // shared memory of an SM for rings

// Sums of a and of b over a warp, in every lane: each half of the lanes
// carries one of the two after the first exchange.
__device__ __forceinline__ void warp_sum2(float& a, float& b) {
  const bool upper = (lane_id() & 16) != 0;
  float s = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  const float other = __shfl_xor_sync(0xffffffffu, s, 16);
  a = upper ? other : s;
  b = upper ? s : other;
}

struct RowRing {
  uint32_t data, bars;
  int slot_bytes, row_bytes, dy_at;  // dy_at: where a slot's rows of dy begin
  // One thread: n rows of x, then of dy, into slot i.
  __device__ __forceinline__ void fill(int i, const char* x, int64_t x_stride, const char* dy, int64_t dy_stride, int n) const {
    const uint32_t bar = bars + 8 * i, dst = data + i * slot_bytes;
    mbar_expect(bar, (uint32_t)(2 * n * row_bytes));
    copy(dst, x, x_stride, n, bar);
    copy(dst + dy_at, dy, dy_stride, n, bar);
  }
  __device__ __forceinline__ void copy(uint32_t dst, const char* src, int64_t stride, int n, uint32_t bar) const {
    if (stride == row_bytes) {
      bulk_copy_in(dst, src, n * row_bytes, bar);
    } else {
      for (int r = 0; r < n; ++r) bulk_copy_in(dst + r * row_bytes, src + r * stride, row_bytes, bar);
    }
  }
};

__device__ __forceinline__ uint4 lds_vec(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
  return v;
}

// What a thread does that gave up its wait: the last of the warps' places in
// both buffers of sums, which no warp has, makes all threads' sums NaN from now
// on, and thread 0 waits once more (bounded) for the copies on their way, from
// `slot` on, for rows `step` apart of which `left` are left. Not inline: inside
// the loop it cost the whole kernel 2 to 8 % (8192 x 7168 bf16 68 us alone, with
// it inline 69 to 74).
__device__ __noinline__ bool give_up(float4* last, uint32_t bars, int slot, int slots, uint32_t parity, int64_t left, int64_t step) {
  last[0] = last[kWarp] = make_float4(kNaN, kNaN, kNaN, kNaN);
  if (threadIdx.x == 0)
    for (int i = slot; i < slot + slots - 1 && (i - slot) * step < left; ++i)
      mbar_wait(bars + 8 * (i < slots ? i : i - slots), i < slots ? parity : parity ^ 1);
  return false;
}

// NV vectors a thread, R rows at a time; KEEP: the weights stay in registers;
// FULL: every thread has all its vectors.
template <typename ET, typename WT, int NV, int R, bool KEEP, bool FULL>
__global__ void __maxnreg__(ring_registers<ET>(NV)) bwd_ring_kernel(BwdArgs a, int slots) {
  using L = Lanes<16, ET>;
  constexpr int kE = L::kElems;
  using P = Pack<kE>;
  using T = typename P::T;
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ uint64_t bars[kMaxSlots];
  __shared__ float4 red[2][kWarp];
  const int lane = lane_id(), warp = threadIdx.x / kWarp;
  const int vecs = (int)(a.H / kE), apart = (int)blockDim.x * 16;
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) in[j] = FULL || (int)(threadIdx.x + j * blockDim.x) < vecs;
  const int row_bytes = vecs * 16;
  const RowRing ring{smem_u32(dyn), smem_u32(bars), 2 * R * row_bytes, row_bytes, R * row_bytes};
  if (threadIdx.x == 0) {
    for (int i = 0; i < slots; ++i) mbar_init(ring.bars + 8 * i);
    fence_mbarrier_init();
  }
  for (int i = threadIdx.x; i < 2 * kWarp; i += blockDim.x) red[i / kWarp][i % kWarp] = make_float4(0, 0, 0, 0);
  await_previous_kernel();
  __syncthreads();
  const int64_t x_stride = a.x_stride * Elem<ET>::kBytes, dy_stride = a.dy_stride * Elem<ET>::kBytes;
  const int64_t step = (int64_t)gridDim.x * R, first = (int64_t)blockIdx.x * R;
  auto fill = [&](int i, int64_t row) {
    if (row < a.rows)
      ring.fill(i, static_cast<const char*>(a.x) + row * x_stride, x_stride,
                static_cast<const char*>(a.dy) + row * dy_stride, dy_stride,
                a.rows - row < R ? (int)(a.rows - row) : R);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < slots - 1; ++i) fill(i, first + i * step);
  auto cols = [&](int j, T (&c)[P::N]) {
    load_cols<WT, kE>(in[j] ? a.weight : nullptr, (int64_t)(threadIdx.x + j * blockDim.x) * kE, 1.0f, c);
  };
  T w[KEEP ? NV : 1][P::N], aw[NV][P::N], ab[NV][P::N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (KEEP) cols(j, w[j]);
#pragma unroll
    for (int q = 0; q < P::N; ++q) aw[j][q] = ab[j][q] = P::splat(0.0f);
  }
  const float inv_h = 1.0f / (float)a.H;
  int slot = 0, buf = 0;
  uint32_t parity = 0;
  bool ok = true;
  char* out = static_cast<char*>(a.dx) + first * row_bytes + threadIdx.x * 16;
  for (int64_t row = first; row < a.rows; row += step, out += step * row_bytes) {
    const bool second = R > 1 && row + 1 < a.rows;
    float s0[R], s1[R], mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = r == 0 || second ? __ldg(a.mean + row + r) : 0.0f;
      rstd[r] = r == 0 || second ? __ldg(a.rstd + row + r) : 0.0f;
    }
    ok = ok && ((a.waits && mbar_wait(ring.bars + 8 * slot, parity)) ||
                give_up(&red[0][kWarp - 1], ring.bars, slot, slots, parity, a.rows - row, step));
    const uint32_t at = ring.data + slot * ring.slot_bytes + threadIdx.x * 16;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const T m2 = P::splat(mean[r]), r2 = P::splat(rstd[r]);
      T t0 = P::splat(0.0f), t1 = t0;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const bool there = in[j] && (r == 0 || second);
        const uint4 x = there ? lds_vec(at + r * row_bytes + j * apart) : make_uint4(0, 0, 0, 0);
        const uint4 d = there ? lds_vec(at + (R + r) * row_bytes + j * apart) : make_uint4(0, 0, 0, 0);
        T(&wj)[P::N] = w[KEEP ? j : 0];
        if (!KEEP) cols(j, wj);
#pragma unroll
        for (int q = 0; q < P::N; ++q) {
          const T dy = P::template get<ET>(d, q);
          const T xhat = P::mul(P::sub(P::template get<ET>(x, q), m2), r2);
          const T v = P::mul(dy, wj[q]);
          t0 = P::add(t0, v);
          t1 = P::fma(v, xhat, t1);
          aw[j][q] = P::fma(dy, xhat, aw[j][q]);  // a row past the last has dy = 0
          ab[j][q] = P::add(ab[j][q], dy);
        }
      }
      s0[r] = P::sum(t0);
      s1[r] = P::sum(t1);
    }
    auto sums = [&] {
      if constexpr (R == 1) {
        warp_sum2(s0[0], s1[0]);
      } else {
        warp_sum2(s0[0], s0[1]);
        warp_sum2(s1[0], s1[1]);
      }
    };
    sums();
    if (lane == 0) red[buf][warp] = make_float4(s0[0], s0[R - 1], s1[0], s1[R - 1]);
    __syncthreads();
    const float4 p = red[buf][lane];
    buf ^= 1;
    if (threadIdx.x == 0 && ok) {  // everybody has read the slot before this one
      fence_async_shared();
      fill(slot == 0 ? slots - 1 : slot - 1, row + (slots - 1) * step);
    }
    s0[R - 1] = p.y;
    s1[R - 1] = p.w;
    s0[0] = p.x;
    s1[0] = p.z;
    sums();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r == 1 && !second) break;
      const T m2 = P::splat(mean[r]), r2 = P::splat(ok ? rstd[r] : kNaN);
      const T c0 = P::splat(s0[r] * inv_h), c1 = P::splat(-s1[r] * inv_h);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!in[j]) break;
        const uint4 x = lds_vec(at + r * row_bytes + j * apart), d = lds_vec(at + (R + r) * row_bytes + j * apart);
        T(&wj)[P::N] = w[KEEP ? j : 0];
        if (!KEEP) cols(j, wj);
        float o[kE];
#pragma unroll
        for (int q = 0; q < P::N; ++q) {
          const T xhat = P::mul(P::sub(P::template get<ET>(x, q), m2), r2);
          const T v = P::mul(P::template get<ET>(d, q), wj[q]);
          P::put(P::mul(P::fma(xhat, c1, P::sub(v, c0)), r2), o + 2 * q);
        }
        st_stream(reinterpret_cast<uint4*>(out + r * row_bytes + j * apart), L::pack(o));
      }
    }
    if (++slot == slots) {
      slot = 0;
      parity ^= 1;
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!in[j]) break;
    float* pw = a.partial + (int64_t)blockIdx.x * a.H + (int64_t)(threadIdx.x + j * blockDim.x) * kE;
    float* pb = pw + (int64_t)gridDim.x * a.H;
#pragma unroll
    for (int q = 0; q < P::N; ++q) {
      float v[2];
      P::put(aw[j][q], v);
      if (!ok) v[0] = v[1] = kNaN;
      *reinterpret_cast<float2*>(pw + 2 * q) = make_float2(v[0], v[1]);
      P::put(ab[j][q], v);
      if (!ok) v[0] = v[1] = kNaN;
      *reinterpret_cast<float2*>(pb + 2 * q) = make_float2(v[0], v[1]);
    }
  }
}

// ------------------------------------------- packed rows off 16 bytes
//
// Rows that follow one another without a gap, of a length that 16 bytes do not
// divide: eight of them together are a multiple of 16 bytes whatever their
// length, so a CTA copies eight in at once (and dy's), works on them element
// by element in shared memory, and copies the results out the same way. First
// a warp takes a row, for its sums, then a thread takes columns, with their
// weights and sums over rows in registers. CTAs overlap their copies with one
// another, two of them at least on an SM. Element loads from global memory
// have too few bytes in flight: forward and backward 96 and 157 us, 55 and 112
// so (58441 x 1001 bf16). fp32 rows have twice the bytes and gain less: 49 and
// 85 against 41 and 95 (29220 x 1001), 70 and 116 against 51 and 77 (100000 x
// 257). Few rows want a CTA each: backward 8.6 against 9.0 at 600 x 1001 bf16,
// 10.2 against 9.8 at 1216. One CTA an SM: backward 146 against 173 (14000 x
// 4095 bf16).

constexpr int kChunk = 8;  // rows
constexpr int kChunkThreads = kChunk * kWarp;
constexpr int kChunkCols = 16;  // columns of a thread at most

template <typename ET> __device__ __forceinline__ float to_float(ET v) { return static_cast<float>(v); }
template <typename ET> __device__ __forceinline__ ET from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The elements of n that fill whole 16 bytes.
template <typename ET> __device__ __forceinline__ int whole16(int n) { return n / Lanes<16, ET>::kElems * Lanes<16, ET>::kElems; }

template <typename ET, typename WT, int NC> __global__ void __launch_bounds__(kChunkThreads) fwd_chunk_kernel(FwdArgs a) {
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ uint64_t bar;
  __shared__ float2 stat[kChunk];
  ET* const sm = reinterpret_cast<ET*>(dyn);
  const int t = threadIdx.x, lane = lane_id(), warp = t / kWarp, H = (int)a.H;
  if (t == 0) {
    mbar_init(smem_u32(&bar));
    fence_mbarrier_init();
  }
  await_previous_kernel();
  __syncthreads();
  float w[NC], b[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = t + j * kChunkThreads;
    w[j] = a.weight != nullptr && c < H ? load1<WT>(a.weight, c) : 1.0f;
    b[j] = a.bias != nullptr && c < H ? load1<WT>(a.bias, c) : 0.0f;
  }
  const float inv_h = 1.0f / (float)H;
  uint32_t parity = 0;
  bool ok = true;
  for (int64_t row = (int64_t)blockIdx.x * kChunk; row < a.rows; row += (int64_t)gridDim.x * kChunk) {
    const int rows = a.rows - row < kChunk ? (int)(a.rows - row) : kChunk, n = rows * H, m = whole16<ET>(n);
    const ET* x = static_cast<const ET*>(a.x) + row * H;
    if (t == 0) {
      bulk_wait_all();  // the last results have left shared memory
      if (ok) bulk_load(smem_u32(dyn), x, (uint32_t)(m * sizeof(ET)), smem_u32(&bar));
    }
    // Bounded; a copy that does not land gets a second wait, then the row's
    // sums are NaN, whichever of its threads gave up.
    ok = ok && ((a.waits && mbar_wait(smem_u32(&bar), parity)) || (mbar_wait(smem_u32(&bar), parity), false));
    parity ^= 1;
    if (m < n) {
      if (t < n - m) sm[m + t] = x[m + t];
      __syncthreads();
    }
    if (warp < rows) {
      const ET* r = sm + warp * H;
      float s[1] = {0.0f}, d[1] = {0.0f};
#pragma unroll 8
      for (int c = lane; c < H; c += kWarp) s[0] += to_float(r[c]);
      if (!ok) s[0] = kNaN;
      lane_sum<1, kWarp>(s);
      const float mean = s[0] * inv_h;
#pragma unroll 8
      for (int c = lane; c < H; c += kWarp) {
        const float e = to_float(r[c]) - mean;
        d[0] = fmaf(e, e, d[0]);
      }
      lane_sum<1, kWarp>(d);
      const float rstd = rsqrtf(d[0] * inv_h + a.eps);
      if (lane == 0) {
        stat[warp] = make_float2(mean, rstd);
        if (a.mean != nullptr) a.mean[row + warp] = mean;
        if (a.rstd != nullptr) a.rstd[row + warp] = rstd;
      }
    }
    __syncthreads();
    for (int r = 0; r < rows; ++r) {
      const float2 st = stat[r];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = t + j * kChunkThreads;
        if (c < H) sm[r * H + c] = from_float<ET>(fmaf((to_float(sm[r * H + c]) - st.x) * st.y, w[j], b[j]));
      }
    }
    fence_async_shared();
    __syncthreads();
    ET* y = static_cast<ET*>(a.y) + row * H;
    if (t == 0) {
      bulk_store(y, smem_u32(dyn), (uint32_t)(m * sizeof(ET)));
      bulk_commit();
    }
    if (t < n - m) y[m + t] = sm[m + t];
  }
  if (t == 0) bulk_wait_all();
}

template <typename ET, typename WT, int NC> __global__ void __launch_bounds__(kChunkThreads) bwd_chunk_kernel(BwdArgs a) {
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ uint64_t bar;
  __shared__ float4 stat[kChunk];
  const int t = threadIdx.x, lane = lane_id(), warp = t / kWarp, H = (int)a.H;
  ET *const sx = reinterpret_cast<ET*>(dyn), *const sd = sx + kChunk * H;
  if (t == 0) {
    mbar_init(smem_u32(&bar));
    fence_mbarrier_init();
  }
  await_previous_kernel();
  __syncthreads();
  float w[NC], aw[NC], ab[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = t + j * kChunkThreads;
    w[j] = a.weight != nullptr && c < H ? load1<WT>(a.weight, c) : 1.0f;
    aw[j] = ab[j] = 0.0f;
  }
  const float inv_h = 1.0f / (float)H;
  uint32_t parity = 0;
  bool ok = true;
  for (int64_t row = (int64_t)blockIdx.x * kChunk; row < a.rows; row += (int64_t)gridDim.x * kChunk) {
    const int rows = a.rows - row < kChunk ? (int)(a.rows - row) : kChunk, n = rows * H, m = whole16<ET>(n);
    const ET *x = static_cast<const ET*>(a.x) + row * H, *dy = static_cast<const ET*>(a.dy) + row * H;
    if (t == 0) {
      bulk_wait_all();
      const uint32_t bytes = (uint32_t)(m * sizeof(ET)), at = smem_u32(&bar);
      if (ok) {
        mbar_expect(at, 2 * bytes);
        bulk_copy_in(smem_u32(sx), x, bytes, at);
        bulk_copy_in(smem_u32(sd), dy, bytes, at);
      }
    }
    float mean = 0.0f, rstd = 0.0f;
    if (warp < rows) {
      mean = __ldg(a.mean + row + warp);
      rstd = __ldg(a.rstd + row + warp);
    }
    ok = ok && ((a.waits && mbar_wait(smem_u32(&bar), parity)) || (mbar_wait(smem_u32(&bar), parity), false));
    parity ^= 1;
    if (m < n) {
      if (t < n - m) {
        sx[m + t] = x[m + t];
        sd[m + t] = dy[m + t];
      }
      __syncthreads();
    }
    if (warp < rows) {
      const ET *rx = sx + warp * H, *rd = sd + warp * H;
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 8
      for (int c = lane; c < H; c += kWarp) {
        const float v = to_float(rd[c]) * (a.weight != nullptr ? load1<WT>(a.weight, c) : 1.0f);
        s0 += v;
        s1 = fmaf(v, (to_float(rx[c]) - mean) * rstd, s1);
      }
      if (!ok) s0 = s1 = kNaN;
      warp_sum2(s0, s1);
      if (lane == 0) stat[warp] = make_float4(mean, rstd, s0 * inv_h, -s1 * inv_h);
    }
    __syncthreads();
    for (int r = 0; r < rows; ++r) {
      const float4 st = stat[r];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = t + j * kChunkThreads;
        if (c < H) {
          const float dyv = to_float(sd[r * H + c]), xhat = (to_float(sx[r * H + c]) - st.x) * st.y;
          aw[j] = fmaf(dyv, xhat, aw[j]);
          ab[j] += dyv;
          sx[r * H + c] = from_float<ET>(fmaf(xhat, st.w, fmaf(dyv, w[j], -st.z)) * st.y);
        }
      }
    }
    fence_async_shared();
    __syncthreads();
    ET* dx = static_cast<ET*>(a.dx) + row * H;
    if (t == 0) {
      bulk_store(dx, smem_u32(sx), (uint32_t)(m * sizeof(ET)));
      bulk_commit();
    }
    if (t < n - m) dx[m + t] = sx[m + t];
  }
  if (t == 0) bulk_wait_all();
  if (a.partial == nullptr) return;
  float* pw = a.partial + (int64_t)blockIdx.x * H;
  float* pb = pw + (int64_t)gridDim.x * H;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = t + j * kChunkThreads;
    if (c < H) {
      pw[c] = ok ? aw[j] : kNaN;
      pb[c] = ok ? ab[j] : kNaN;
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
    row_sum<1, 0>(s, red, buf);
    const float mean = s[0] * inv_h;
    s[0] = 0.0f;
    for (int64_t c = threadIdx.x; c < a.H; c += blockDim.x) {
      const float d = load1<ET>(x, c) - mean;
      s[0] += d * d;
    }
    row_sum<1, 0>(s, red, buf);
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
    row_sum<2, 0>(s, red, buf);
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

// Adds the CTAs' partial sums: 32 columns per CTA, its NW warps each a share
// of the parts. blockIdx.y: 0 dweight, 1 dbias. Few columns make few CTAs: 32
// warps then, with ten loads ahead (the whole backward pass, replayed from a
// CUDA graph, 1531 x 1001 fp32, 9.2 us, with 16 warps and four 10.4; 4000 x 1000
// bf16 12.1 and 15.9), 16 where the columns alone fill the chip (8192 x 7168:
// 67.4, with 32 69.6).
constexpr int64_t kFewCols = 2048;
template <typename WT, int NW>
__global__ void __launch_bounds__(NW * kWarp) cols_kernel(const float* __restrict__ partial, int parts, int64_t H,
                                                          WT* dweight, WT* dbias) {
  __shared__ float red[NW][kWarp];
  await_previous_kernel();
  WT* out = blockIdx.y == 0 ? dweight : dbias;
  if (out == nullptr) return;
  const int lane = lane_id(), warp = threadIdx.x / kWarp;
  const int64_t c = (int64_t)blockIdx.x * kWarp + lane;
  float s = 0.0f;
  if (c < H) {
    const float* p = partial + (int64_t)blockIdx.y * parts * H + c;
#pragma unroll(NW == 32 ? 10 : 4)
    for (int g = warp; g < parts; g += NW) s += __ldcg(p + (int64_t)g * H);
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < H) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) t += red[w][lane];
    store1(out, c, t);
  }
}

// ------------------------------------------------------------------ host

constexpr int kMinParts = 304;    // CTAs of the backward pass, each with a row of partial column sums,
constexpr int kMaxParts = 2432;   // more of them for shorter rows:
constexpr int64_t kPartElems = (int64_t)304 * 8192;
constexpr int64_t kPartRows = 4;  // rows of a CTA at least, where there are kMinParts of them (4000 x 1000 bf16:
                                  // 12.0 us, with 1.6 rows each 16.4)

int64_t bwd_parts(int64_t rows, int64_t H) {
  int64_t most = kPartElems / H;
  const int64_t few = rows / kPartRows < kMinParts ? kMinParts : rows / kPartRows;
  if (most > few) most = few;
  most = most < kMinParts ? kMinParts : (most > kMaxParts ? kMaxParts : most);
  return rows < most ? rows : most;
}

int cta_threads(int64_t vecs, int nv) { return (int)(((vecs + nv - 1) / nv + kWarp - 1) / kWarp * kWarp); }

// Grid, threads and slots of the ring kernel for rows of `vecs` vectors, nv a
// thread and r rows at a time; false where they are too short or long for it.
struct RingShape {
  int threads, grid, slots;
  size_t smem;
};
bool ring_shape(int64_t vecs, int nv, int r, int registers, int threads, int64_t rows, int64_t most, RingShape* z) {
  z->threads = cta_threads(vecs, nv);
  if (vecs <= kWarp || z->threads > threads) return false;
  int per_sm = 65536 / ((registers + 7) / 8 * 8) / z->threads;
  if (per_sm > 16) per_sm = 16;
  if (per_sm < 1) per_sm = 1;
  const int64_t slot = 2 * r * vecs * 16, n = kRingSm / per_sm / slot;
  z->slots = (int)(n < kMaxSlots ? n : kMaxSlots);
  z->smem = (size_t)(z->slots * slot);
  int64_t g = (int64_t)num_sms() * per_sm;
  if (g > most) g = most;
  const int64_t work = (rows + r - 1) / r;
  z->grid = (int)(work < g ? work : g);
  return z->slots >= 2;
}

// Whether the chunk kernels take the rows: packed, enough of them for every SM,
// and `arrays` chunks in at most `most` bytes of shared memory.
template <typename ET> bool chunks_ok(int64_t H, int64_t rows, int arrays, int64_t most, const int64_t* strides, const void* const* ptrs) {
  bool ok = H > kChunkThreads && H <= kChunkCols * kChunkThreads && arrays * kChunk * H * Elem<ET>::kBytes <= most &&
            rows >= kChunk * (int64_t)num_sms();
  for (int i = 0; i < arrays; ++i) ok = ok && strides[i] == H;
  for (int i = 0; i <= arrays; ++i) ok = ok && aligned(ptrs[i], 16);
  return ok;
}

template <typename ET, typename WT, int NC> int go_fwd_chunk(const FwdArgs& a, cudaStream_t s) {
  if constexpr (NC > 4) {
    if (a.H <= NC / 2 * kChunkThreads) return go_fwd_chunk<ET, WT, NC / 2>(a, s);
  }
  static std::atomic<bool> raised[kSmemDevices];
  auto k = fwd_chunk_kernel<ET, WT, NC>;
  const size_t smem = (size_t)kChunk * a.H * Elem<ET>::kBytes;
  if (!allow_smem(k, raised)) return MOE_ERR_CUDA;
  launch(k, grid_for(k, kChunkThreads, smem, (a.rows + kChunk - 1) / kChunk), kChunkThreads, smem, s, a);
  return check_launch();
}

template <typename ET, typename WT, int NC> int go_bwd_chunk(const BwdArgs& a, int* parts, cudaStream_t s) {
  if constexpr (NC > 4) {
    if (a.H <= NC / 2 * kChunkThreads) return go_bwd_chunk<ET, WT, NC / 2>(a, parts, s);
  }
  static std::atomic<bool> raised[kSmemDevices];
  auto k = bwd_chunk_kernel<ET, WT, NC>;
  const size_t smem = 2 * (size_t)kChunk * a.H * Elem<ET>::kBytes;
  if (!allow_smem(k, raised)) return MOE_ERR_CUDA;
  const int64_t most = bwd_parts(a.rows, a.H), work = (a.rows + kChunk - 1) / kChunk;
  *parts = grid_for(k, kChunkThreads, smem, work < most ? work : most);
  launch(k, *parts, kChunkThreads, smem, s, a);
  return check_launch();
}

template <int VB, typename ET, typename WT, int NV, int LPR, int DEPTH, int MAXT = kMaxThreads>
int go_fwd(const FwdArgs& a, cudaStream_t s) {
  const int threads = LPR ? kRowWarps * kWarp : cta_threads(a.H / Lanes<VB, ET>::kElems, NV);
  constexpr int kRows = LPR ? kRowWarps * (kWarp / (LPR ? LPR : 1)) : 1;
  auto go = [&](auto k) {
    launch(k, grid_for(k, threads, 0, (a.rows + kRows - 1) / kRows), threads, 0, s, a);
    return check_launch();
  };
  if constexpr (LPR == 0 && VB == 16 && MAXT == 256) {
    if (a.H / Lanes<VB, ET>::kElems == (int64_t)threads * NV) return go(fwd_kernel<VB, ET, WT, NV, LPR, DEPTH, MAXT, true>);
  }
  return go(fwd_kernel<VB, ET, WT, NV, LPR, DEPTH, MAXT, false>);
}

// Vectors of a row decide: lanes of a warp up to 128 of them, a CTA beyond.
template <int VB, typename ET, typename WT> int dispatch_fwd(const FwdArgs& a, cudaStream_t s) {
  const int64_t vecs = a.H / Lanes<VB, ET>::kElems;
  if (vecs <= 8) return go_fwd<VB, ET, WT, 1, 8, 4>(a, s);
  if (vecs <= 16) return go_fwd<VB, ET, WT, 1, 16, 4>(a, s);
  if (vecs <= 32) return go_fwd<VB, ET, WT, 1, 32, 4>(a, s);
  if (vecs <= 64) return go_fwd<VB, ET, WT, 2, 32, 2>(a, s);
  if (vecs <= 128) return go_fwd<VB, ET, WT, 4, 32, 1>(a, s);
  if constexpr (VB == 16) {
    if (vecs <= 4 * 256) return go_fwd<VB, ET, WT, 4, 0, 1, 256>(a, s);
    if (vecs <= 4 * kMaxThreads) return go_fwd<VB, ET, WT, 4, 0, 1>(a, s);
  } else {
    if (vecs <= 8 * kMaxThreads) return go_fwd<VB, ET, WT, 8, 0, 2>(a, s);
    if (vecs <= 16 * kMaxThreads) return go_fwd<VB, ET, WT, 16, 0, 1>(a, s);
  }
  auto k = fwd_long_kernel<ET, WT>;
  launch(k, grid_for(k, 512, 0, a.rows), 512, 0, s, a);
  return check_launch();
}

template <int VB, typename ET, typename WT, int NV, int LPR, int DEPTH, int MAXT = kMaxThreads>
int go_bwd(const BwdArgs& a, int* parts, cudaStream_t s) {
  const int threads = LPR ? kRowWarps * kWarp : cta_threads(a.H / Lanes<VB, ET>::kElems, NV);
  constexpr int kRows = LPR ? kRowWarps * (kWarp / (LPR ? LPR : 1)) : 1;
  const int64_t most = bwd_parts(a.rows, a.H), work = (a.rows + kRows - 1) / kRows;
  const size_t smem = LPR ? sizeof(float) * 2 * NV * LPR * Lanes<VB, ET>::kElems : 0;
  auto k = bwd_kernel<VB, ET, WT, NV, LPR, DEPTH, MAXT>;
  *parts = grid_for(k, threads, smem, work < most ? work : most);
  launch(k, *parts, threads, smem, s, a);
  return check_launch();
}

template <typename ET, typename WT, int NV, int R, bool KEEP, bool FULL = false>
int go_ring(const BwdArgs& a, int* parts, cudaStream_t s) {
  static std::atomic<bool> raised[kSmemDevices];
  RingShape z;
  const int64_t vecs = a.H / Lanes<16, ET>::kElems;
  if constexpr (!FULL) {
    if (vecs == (int64_t)cta_threads(vecs, NV) * NV) return go_ring<ET, WT, NV, R, KEEP, true>(a, parts, s);
  }
  auto k = bwd_ring_kernel<ET, WT, NV, R, KEEP, FULL>;
  if (!ring_shape(vecs, NV, R, ring_registers<ET>(NV), ring_threads<ET>(NV), a.rows, bwd_parts(a.rows, a.H), &z) ||
      !allow_smem(k, raised))
    return MOE_ERR_CUDA;
  *parts = z.grid;
  launch(k, z.grid, z.threads, z.smem, s, a, z.slots);
  return check_launch();
}

template <int VB, typename ET, typename WT> int dispatch_bwd(const BwdArgs& a, int* parts, cudaStream_t s) {
  const int64_t vecs = a.H / Lanes<VB, ET>::kElems;
  if (vecs <= 8) return go_bwd<VB, ET, WT, 1, 8, 2>(a, parts, s);
  if (vecs <= 16) return go_bwd<VB, ET, WT, 1, 16, 2>(a, parts, s);
  if (vecs <= 32) return go_bwd<VB, ET, WT, 1, 32, 2>(a, parts, s);
  if constexpr (VB == 16) {
    if (vecs <= 2 * kRingThreads) return go_ring<ET, WT, 2, 2, true>(a, parts, s);
    if constexpr (Elem<ET>::kBytes == 2) {
      if (vecs <= 4 * kRingThreads) return go_ring<ET, WT, 4, 1, false>(a, parts, s);
    } else {
      if (vecs <= 2 * kMaxThreads) return go_bwd<VB, ET, WT, 2, 0, 1>(a, parts, s);
      if (vecs <= kRingSm / 64) return go_ring<ET, WT, 4, 1, false>(a, parts, s);  // two slots
    }
  } else {
    if (vecs <= 4 * kMaxThreads) return go_bwd<VB, ET, WT, 4, 0, 2>(a, parts, s);
    if (vecs <= 8 * kMaxThreads) return go_bwd<VB, ET, WT, 8, 0, 1>(a, parts, s);
  }
  auto k = bwd_long_kernel<ET, WT>;
  launch(k, grid_for(k, 512, 0, a.rows), 512, 0, s, a);
  *parts = (int)(a.rows < 32 ? a.rows : 32);
  if (a.partial != nullptr)
    launch(bwd_long_cols_kernel<ET>, dim3((unsigned)((a.H + 255) / 256), (unsigned)*parts), 256, 0, s, a);
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

int row_waits() { return test_give_up().load(std::memory_order_relaxed) & kGiveUpRows ? 0 : 1; }

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
  const void* ptrs[] = {a.x, a.y};
  constexpr int kCols = 16 / Elem<ET>::kBytes * Elem<WT>::kBytes;  // of the weights beside 16 bytes of a row
  if (rows_by_16<ET>(a.H, &a.x_stride, 1, ptrs, 2) && aligned(a.weight, kCols) && aligned(a.bias, kCols))
    return dispatch_fwd<16, ET, WT>(a, s);
  if (chunks_ok<ET>(a.H, a.rows, 1, kRingSm / 2, &a.x_stride, ptrs)) return go_fwd_chunk<ET, WT, kChunkCols>(a, s);
  return dispatch_fwd<Elem<ET>::kBytes, ET, WT>(a, s);
}

template <typename ET, typename WT> int run_bwd(BwdArgs a, void* dweight, void* dbias, cudaStream_t s) {
  if (a.rows < 2) a.x_stride = a.dy_stride = a.H;
  int parts = 0, rc = MOE_OK;
  if (a.rows > 0) {
    const int64_t strides[] = {a.x_stride, a.dy_stride};
    const void* ptrs[] = {a.x, a.dy, a.dx};
    if (rows_by_16<ET>(a.H, strides, 2, ptrs, 3) && aligned(a.weight, 16 / Elem<ET>::kBytes * Elem<WT>::kBytes))
      rc = dispatch_bwd<16, ET, WT>(a, &parts, s);
    else if (chunks_ok<ET>(a.H, a.rows, 2, Elem<ET>::kBytes == 2 ? kRingSm / 2 : kRingSm / 6, strides, ptrs))
      rc = go_bwd_chunk<ET, WT, kChunkCols>(a, &parts, s);
    else
      rc = dispatch_bwd<Elem<ET>::kBytes, ET, WT>(a, &parts, s);
  }
  if (rc != MOE_OK || (dweight == nullptr && dbias == nullptr)) return rc;
  const dim3 grid((unsigned)((a.H + kWarp - 1) / kWarp), 2);
  auto go = [&](auto k, int threads) {
    launch(k, grid, threads, 0, s, (const float*)a.partial, parts, a.H, static_cast<WT*>(dweight), static_cast<WT*>(dbias));
  };
  if (a.H <= kFewCols)
    go(cols_kernel<WT, 32>, 32 * kWarp);
  else
    go(cols_kernel<WT, 16>, 16 * kWarp);
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
  const FwdArgs a{x, weight, bias, y, mean, rstd, x_stride, rows, H, eps, row_waits()};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MOE_F32) return wdtype == MOE_F32 ? run_fwd<float, float>(a, s) : run_fwd<float, __nv_bfloat16>(a, s);
  return wdtype == MOE_F32 ? run_fwd<__nv_bfloat16, float>(a, s) : run_fwd<__nv_bfloat16, __nv_bfloat16>(a, s);
}

extern "C" size_t moe_layer_norm_bwd_workspace_size(int64_t rows, int64_t H) {
  if (rows < 0 || H < 1) return 0;
  return (size_t)bwd_parts(rows < 1 ? 1 : rows, H) * 2 * (size_t)H * sizeof(float);
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
                  dy_stride, x_stride, rows, H, row_waits()};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MOE_F32)
    return wdtype == MOE_F32 ? run_bwd<float, float>(a, dweight, dbias, s)
                             : run_bwd<float, __nv_bfloat16>(a, dweight, dbias, s);
  return wdtype == MOE_F32 ? run_bwd<__nv_bfloat16, float>(a, dweight, dbias, s)
                           : run_bwd<__nv_bfloat16, __nv_bfloat16>(a, dweight, dbias, s);
}
