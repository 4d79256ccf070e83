// Attention of one new token of every sequence over a key-value cache in pages:
//   s_j = scale * q . k_j,  out = sum_j softmax(s)_j v_j
//
// Bound by HBM: every key and value of the cache is read once, for 2 * group
// multiply-adds an element (group: query heads that share a kv head).
//
// One pass with a running maximum and sum: for each tile of keys m' = max(m, max s),
// l' = l 2^(m - m') + sum 2^(s - m'), o' = o 2^(m - m') + sum 2^(s - m') v, with s in
// units of log 2. The tiles of all sequences (16 tokens of one kv head) are one
// long line, cut into equal ranges: a warp takes a range of one head, so long
// sequences are split over many warps, short ones share one, and every SM gets
// the same number of bytes whatever the lengths are. A sequence inside one range is
// finished by its warp; the parts of the others are left in the workspace as
// (o, m, l) and joined by a second kernel in the order of the ranges. Warps work
// alone, each with its own ring of asynchronous copies: no barrier in the loop.
// Neighbouring warps take neighbouring heads of the same range, so that an SM
// reads whole rows of a page where heads lie side by side.
#include <math.h>

#include <atomic>

#include "block_common.h"
#include "bulk.cuh"
#include "common.cuh"
#include "moe_decode.h"
#include "vec_math.cuh"

namespace moe {
namespace {

constexpr int kTile = 16;      // tokens of a tile, the unit of the ranges
constexpr int kSmWarps = 8;    // warps of an SM: a CTA of eight, one an SM
constexpr int kMinTiles = 2;   // of a range, where there are fewer tiles than warps
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Quotients by a divisor known at launch, for numerators below 2^31: with
// s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1, n / d = (mulhi(n, m) + n) >> s
// (Granlund and Montgomery, Division by Invariant Integers, 1994).
struct Divisor {
  uint32_t d, m, s;
  Divisor() : Divisor(1) {}
  explicit Divisor(uint32_t by) : d(by), m(0), s(0) {
    while ((1ull << s) < by) ++s;
    m = (uint32_t)(((1ull << 32) * ((1ull << s) - by)) / by + 1);
  }
  __device__ __forceinline__ uint32_t of(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};

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
  int32_t seqs, width, heads, kv_heads, group, D;
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
__device__ __forceinline__ int ranges_of(const AttendArgs& a, int total) {
  const int most = total / kMinTiles;
  return most < a.ranges ? (most < 1 ? 1 : most) : a.ranges;
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
  __device__ __forceinline__ void enter(const AttendArgs& a) {
    span_of(a, b, first, n);
    tiles = (n - first + kTile - 1) / kTile;
  }
  __device__ __forceinline__ void next(const AttendArgs& a) {  // there is a next tile
    if (++tile < tiles) return;
    tile = 0;
    do {
      ++b;
      enter(a);
    } while (tiles == 0);
  }
};

// The joining kernel may start: it waits for this one before it reads what it left.
__device__ __forceinline__ void start_next_kernel() { asm volatile("griddepcontrol.launch_dependents;"); }

// The CTA's view of the line: prefix[t] tiles in front of the sequences of thread t.
__device__ __forceinline__ int line_prefix(const AttendArgs& a, int* prefix, int* s_warp) {
  const int t = threadIdx.x, chunk = (a.seqs + blockDim.x - 1) / blockDim.x;
  int mine = 0;
  for (int b = t * chunk; b < a.seqs && b < (t + 1) * chunk; ++b) {
    if (blockIdx.x == 0 && (a.lengths[b] < 0 || a.lengths[b] > a.max_tokens)) flag_status(a.status, MOE_STATUS_BAD_INDEX);
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
  while (c.tile >= c.tiles) {
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

template <typename ET> __device__ __forceinline__ float to_float(ET v);
template <> __device__ __forceinline__ float to_float<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Heads' rows on the ordinary cores, in fp32: a warp takes 8 keys at a time.
// Scores: lane (key, quarter) takes the fourth of the key's elements that
// `quarter` says, in pieces of four, for all GM heads; values: a lane owns
// pieces of four of a row's elements for all heads.
template <typename ET, int GM, int NC>
__global__ void __launch_bounds__(kSmWarps * kWarp, 1) attend_rows_kernel(const AttendArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_prefix[kSmWarps * kWarp], s_warp[kSmWarps];
  constexpr int kKeys = 8;
  await_previous_kernel();
  start_next_kernel();
  const int lane = lane_id(), warp = threadIdx.x / kWarp;
  const int total = line_prefix(a, s_prefix, s_warp);
  const int HV = a.kv_heads * a.parts, gw = blockIdx.x * kSmWarps + warp;
  const int r = gw / HV, hv = gw - r * HV, kv = hv / a.parts, part = hv - kv * a.parts;
  if (total == 0) return;
  const int ranges = ranges_of(a, total);
  if (r >= ranges) return;
  const int lo = range_begin(r, ranges, total), hi = range_begin(r + 1, ranges, total);
  if (lo >= hi) return;
  Cursor c = find_tile(a, s_prefix, lo);

  const int D = a.D, pieces = (D + 3) / 4;
  const int pitch = (((pieces + 3) / 4) * 4 + ((((pieces + 3) / 4) & 1) ? 0 : 4)) * 4;  // floats; 64 bytes off a multiple of 128
  float* ks = reinterpret_cast<float*>(smem) + (size_t)warp * (2 * kKeys * pitch + GM * pitch + GM * kKeys);
  float* vs = ks + kKeys * pitch;
  float* qs = vs + kKeys * pitch;
  float* ps = qs + GM * pitch;
  for (int i = lane; i < 2 * kKeys * pitch + GM * pitch; i += kWarp) ks[i] = 0.0f;  // what lies behind D stays zero
  __syncwarp();

  const int h0 = kv * a.group + part * GM, count = min(GM, a.group - part * GM);
  const int key = lane >> 2, quarter = lane & 3;
  float m[GM], l[GM], o[GM][NC][4];
  bool fresh = true;
  int first_tile = c.tile;
  int64_t x = lo;
  while (true) {
    if (fresh) {
      fresh = false;
      first_tile = c.tile;
      for (int h = 0; h < count; ++h) {
        const ET* row = reinterpret_cast<const ET*>(a.q + c.b * a.q_row + (h0 + h) * a.q_head);
        for (int d = lane; d < D; d += kWarp) qs[h * pitch + d] = to_float(row[d]) * a.scale;
      }
#pragma unroll
      for (int h = 0; h < GM; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.0f;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[h][j][e] = 0.0f;
      }
      __syncwarp();
    }
    const int mine = lane & (kTile - 1);
    const int64_t off = row_offset(a, c, mine, page_entry(a, c, mine), kv);
    const int new_row = a.k_new != nullptr ? c.n - 1 - (c.first + c.tile * kTile) : -1;  // of the new token, if in 0 .. 15
    const unsigned valid = __ballot_sync(0xffffffffu, off >= 0) & 0xffffu;
    for (int half = 0; half < 2; ++half) {
      const unsigned bits = valid >> (half * kKeys) & 0xffu;
      if (bits == 0) continue;
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        const int row = half * kKeys + i;
        const int64_t at = __shfl_sync(0xffffffffu, off, row);
        if (at < 0) {
          for (int d = lane; d < D; d += kWarp) ks[i * pitch + d] = vs[i * pitch + d] = 0.0f;
          continue;
        }
        ET* kc = reinterpret_cast<ET*>(a.k + at);
        ET* vc = reinterpret_cast<ET*>(a.v + at);
        if (row == new_row) {
          const ET* kn = reinterpret_cast<const ET*>(a.k_new + c.b * a.kn_row + kv * a.kn_head);
          const ET* vn = reinterpret_cast<const ET*>(a.v_new + c.b * a.vn_row + kv * a.vn_head);
          for (int d = lane; d < D; d += kWarp) {
            const ET kk = kn[d], vv = vn[d];
            if (part == 0) {
              kc[d] = kk;
              vc[d] = vv;
            }
            ks[i * pitch + d] = to_float(kk);
            vs[i * pitch + d] = to_float(vv);
          }
        } else {
          for (int d = lane; d < D; d += kWarp) {
            ks[i * pitch + d] = to_float(kc[d]);
            vs[i * pitch + d] = to_float(vc[d]);
          }
        }
      }
      __syncwarp();
      // Scores of (key, all heads), the same in the four lanes of a key.
      float s[GM];
#pragma unroll
      for (int h = 0; h < GM; ++h) s[h] = 0.0f;
      for (int p = quarter; p < pieces; p += 4) {
        const float4 kk = *reinterpret_cast<const float4*>(ks + key * pitch + 4 * p);
#pragma unroll
        for (int h = 0; h < GM; ++h) {
          const float4 qq = *reinterpret_cast<const float4*>(qs + h * pitch + 4 * p);
          s[h] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, s[h]))));
        }
      }
#pragma unroll
      for (int h = 0; h < GM; ++h) {
        s[h] += __shfl_xor_sync(0xffffffffu, s[h], 1);
        s[h] += __shfl_xor_sync(0xffffffffu, s[h], 2);
        if (!(bits >> key & 1)) s[h] = -INFINITY;
        float t = s[h];
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
        const float now = fmaxf(m[h], t);
        const float base = now == -INFINITY ? 0.0f : now;
        const float keep = exp2f(m[h] - base);
        const float pr = exp2f(s[h] - base);
        m[h] = now;
        l[h] = l[h] * keep + (quarter == 0 ? pr : 0.0f);
        if (quarter == 0) ps[h * kKeys + key] = pr;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[h][j][e] *= keep;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          const int p = lane + j * kWarp;
          if (p < pieces) {
            const float4 vv = *reinterpret_cast<const float4*>(vs + i * pitch + 4 * p);
#pragma unroll
            for (int h = 0; h < GM; ++h) {
              const float pr = ps[h * kKeys + i];
              o[h][j][0] = fmaf(pr, vv.x, o[h][j][0]);
              o[h][j][1] = fmaf(pr, vv.y, o[h][j][1]);
              o[h][j][2] = fmaf(pr, vv.z, o[h][j][2]);
              o[h][j][3] = fmaf(pr, vv.w, o[h][j][3]);
            }
          }
        }
      }
      __syncwarp();
    }
    ++x;
    const bool last = c.tile == c.tiles - 1;
    if (last || x == hi) {
      const bool whole = last && first_tile == 0;
      const int64_t slot = (int64_t)r + c.b;
#pragma unroll
      for (int h = 0; h < GM; ++h) {
        float sum = l[h];
#pragma unroll
        for (int d = 1; d < kWarp; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (h >= count) continue;
        const int64_t head = whole ? (int64_t)c.b * a.heads + h0 + h : slot * a.heads + h0 + h;
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int d = 4 * (lane + j * kWarp) + e;
            if (d >= D) continue;
            if (!whole) {
              a.part_o[head * D + d] = o[h][j][e];
            } else if constexpr (sizeof(ET) == 4) {
              static_cast<float*>(a.out)[head * D + d] = o[h][j][e] * inv;
            } else {
              static_cast<__nv_bfloat16*>(a.out)[head * D + d] = __float2bfloat16_rn(o[h][j][e] * inv);
            }
          }
        if (lane == 0) {
          if (!whole) {
            a.part_ml[head] = make_float2(m[h], sum);
          } else if (a.lse != nullptr) {
            a.lse[head] = sum > 0.0f ? (m[h] + log2f(sum)) * kLn2 : -INFINITY;
          }
        }
      }
      fresh = true;
    }
    if (x == hi) break;
    c.next(a);
  }
}

// ------------------------------------------------- bf16, on the tensor cores

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldmatrix(uint32_t (&f)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3]) : "r"(at));
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&f)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3]) : "r"(at));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Sizes of a variant: DP elements of a padded row (64, 128 or 256), MT tiles of
// 16 query heads (0: eight heads in one).
template <int DP, int MT> struct Mma {
  static constexpr int kHeads = MT == 0 ? 8 : 16 * MT, kTiles = MT == 0 ? 1 : MT;
  static constexpr int kWarps = DP == 256 ? 4 : 8;
  static constexpr int kStageBytes = 2 * kTile * DP * 2;
  static constexpr int kStages = DP == 64 ? 6 : 3;  // 192 KB an SM
  static constexpr size_t kSmem = (size_t)kWarps * kStages * kStageBytes;
};

// S = Q K^T and O += P V by m16n8k16 products: the query heads of a kv head are
// the rows, 16 keys a step. Decoding has few rows, so the products are never
// the bound (16 keys of 128 elements: 32 to 48 instructions in the 350 clocks
// that the SM's share of HBM needs for them). P goes in as two bf16 numbers, the
// second what the first one's rounding left; with eight heads or fewer the
// second takes the rows that they leave empty, and costs nothing.
template <int DP, int MT>
__global__ void __launch_bounds__(Mma<DP, MT>::kWarps * kWarp, 1) attend_mma_kernel(const AttendArgs a) {
  using S = Mma<DP, MT>;
  constexpr int kWarps = S::kWarps, kStages = S::kStages, kTiles = S::kTiles;
  constexpr int kChunks = DP / 8, kRowsPass = kWarp / kChunks, kPasses = kTile / kRowsPass;  // 16-byte pieces of a row
  constexpr int kSteps = DP / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_prefix[kWarps * kWarp], s_warp[kWarps];
  __shared__ unsigned s_mask[kWarps][kStages];
  await_previous_kernel();
  start_next_kernel();
  const int lane = lane_id(), warp = threadIdx.x / kWarp;
  const int total = line_prefix(a, s_prefix, s_warp);
  const int HV = a.kv_heads * a.parts, gw = blockIdx.x * kWarps + warp;
  const int r = gw / HV, hv = gw - r * HV, kv = hv / a.parts, part = hv - kv * a.parts;
  if (total == 0) return;
  const int ranges = ranges_of(a, total);
  if (r >= ranges) return;
  const int lo = range_begin(r, ranges, total), count = range_begin(r + 1, ranges, total) - lo;
  if (count <= 0) return;
  const int D = a.D, h0 = kv * a.group + part * S::kHeads, heads = min(S::kHeads, a.group - part * S::kHeads);
  const uint32_t ring = smem_u32(smem) + warp * kStages * S::kStageBytes;
  if (D < DP) {  // pieces behind D are never copied, and have to be numbers
    uint4* z = reinterpret_cast<uint4*>(smem + (size_t)warp * kStages * S::kStageBytes);
    for (int i = lane; i < kStages * S::kStageBytes / 16; i += kWarp) z[i] = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }

  // Copies of a tile: K then V, 16 rows each, pieces swizzled by the row.
  Cursor in = find_tile(a, s_prefix, lo);
  Cursor at = in;
  int issued = 0, page = page_entry(a, in, lane & (kTile - 1));
  const int chunk = lane % kChunks, sub = lane / kChunks;
  const bool copies = chunk * 8 < D;
  const auto issue = [&]() {
    if (issued < count) {
      const int stage = issued % kStages, row = lane & (kTile - 1);
      int64_t off = row_offset(a, in, row, page, kv);
      const unsigned valid = __ballot_sync(0xffffffffu, off >= 0) & 0xffffu;
      if (lane == 0) s_mask[warp][stage] = valid;
      const int fresh = a.k_new != nullptr ? in.n - 1 - (in.first + in.tile * kTile) : -1;  // the new token's row
      const uint32_t base = ring + stage * S::kStageBytes;
      if (fresh >= 0 && fresh < kTile && (valid >> fresh & 1)) {
        const int64_t to = __shfl_sync(0xffffffffu, off, fresh);
        if (lane == fresh || lane == fresh + kTile) off = -2;
        if (sub == 0 && copies) {
          const char* kn = a.k_new + in.b * a.kn_row + kv * a.kn_head + chunk * 16;
          const char* vn = a.v_new + in.b * a.vn_row + kv * a.vn_head + chunk * 16;
          const uint32_t dst = base + fresh * DP * 2 + ((chunk ^ (fresh & 7)) * 16);
          cp_async16(dst, kn, 16);
          cp_async16(dst + kTile * DP * 2, vn, 16);
          if (part == 0) {
            *reinterpret_cast<uint4*>(a.k + to + chunk * 16) = *reinterpret_cast<const uint4*>(kn);
            *reinterpret_cast<uint4*>(a.v + to + chunk * 16) = *reinterpret_cast<const uint4*>(vn);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int row_i = i * kRowsPass + sub;
        const int64_t from = __shfl_sync(0xffffffffu, off, row_i);
        if (copies && from != -2) {
          const int bytes = from < 0 ? 0 : 16;
          const int64_t o = from < 0 ? 0 : from + chunk * 16;
          const uint32_t dst = base + row_i * DP * 2 + ((chunk ^ (row_i & 7)) * 16);
          cp_async16(dst, a.k + o, bytes);
          cp_async16(dst + kTile * DP * 2, a.v + o, bytes);
        }
      }
      if (++issued < count) {
        in.next(a);
        page = page_entry(a, in, row);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue();

  uint32_t q[kTiles][kSteps][4];
  float o[kTiles][DP / 8][4], m[kTiles][2], l[kTiles][2];
  const int g = lane >> 2, t = lane & 3;
  const int mi = lane >> 3, lr = lane & 7;
  const uint32_t k_at = ((mi >> 1) * 8 + lr) * DP * 2, v_at = ((mi & 1) * 8 + lr) * DP * 2 + kTile * DP * 2;
  bool fresh = true;
  int first_tile = at.tile;
  for (int i = 0; i < count; ++i) {
    if (fresh) {
      fresh = false;
      first_tile = at.tile;
      const char* rows = a.q + at.b * a.q_row;
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int h = u * 16 + g + (e & 1) * 8, d = ks * 16 + t * 2 + (e >> 1) * 8;
            q[u][ks][e] = (MT == 0 && (e & 1)) || h >= heads || d >= D
                              ? 0u : __ldg(reinterpret_cast<const unsigned*>(rows + (h0 + h) * a.q_head + d * 2));
          }
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[u][n][e] = 0.0f;
        m[u][0] = m[u][1] = -INFINITY;
        l[u][0] = l[u][1] = 0.0f;
      }
    }
    cp_wait<kStages - 2>();
    __syncwarp();
    const int stage = i % kStages;
    const unsigned valid = s_mask[warp][stage];
    issue();  // into the stage that the previous tile left
    const uint32_t base = ring + stage * S::kStageBytes;
    float s[kTiles][2][4];
#pragma unroll
    for (int u = 0; u < kTiles; ++u)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[u][n][e] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) {
      uint32_t b[4];
      ldmatrix(b, base + k_at + (((ks * 2 + (mi & 1)) ^ lr) * 16));
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        mma(s[u][0], q[u][ks], b[0], b[1]);
        mma(s[u][1], q[u][ks], b[2], b[3]);
      }
    }
    uint32_t hi[kTiles][4], lo2[kTiles][4];
#pragma unroll
    for (int u = 0; u < kTiles; ++u) {
      constexpr int kRows = MT == 0 ? 1 : 2;  // rows g and g + 8
      float keep[2] = {1.0f, 1.0f};
      bool moved = false;
#pragma unroll
      for (int w = 0; w < kRows; ++w) {
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = s[u][n][2 * w + e];
            x *= a.scale;
            if (valid != 0xffffu && !(valid >> (n * 8 + t * 2 + e) & 1)) x = -INFINITY;
            top = fmaxf(top, x);
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float now = fmaxf(m[u][w], top), from = now == -INFINITY ? 0.0f : now;
        if (now > m[u][w]) {
          moved = true;
          keep[w] = ex2(m[u][w] - from);
          m[u][w] = now;
        }
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = ex2(s[u][n][2 * w] - from), p1 = ex2(s[u][n][2 * w + 1] - from);
          sum += p0 + p1;
          const uint32_t h = pack_bf16x2(p0, p1);
          const uint32_t rest = pack_bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u));
          if constexpr (MT == 0) {
            hi[u][2 * n] = h;
            hi[u][2 * n + 1] = rest;
          } else {
            hi[u][2 * n + w] = h;
            lo2[u][2 * n + w] = rest;
          }
        }
        l[u][w] = l[u][w] * keep[w] + sum;
      }
      if (__any_sync(0xffffffffu, moved)) {
        if constexpr (MT == 0) keep[1] = keep[0];
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) {
          o[u][n][0] *= keep[0];
          o[u][n][1] *= keep[0];
          o[u][n][2] *= keep[1];
          o[u][n][3] *= keep[1];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kSteps; ++c) {
      uint32_t b[4];
      ldmatrix_trans(b, base + v_at + (((c * 2 + (mi >> 1)) ^ lr) * 16));
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        mma(o[u][2 * c], hi[u], b[0], b[1]);
        mma(o[u][2 * c + 1], hi[u], b[2], b[3]);
        if constexpr (MT > 0) {
          mma(o[u][2 * c], lo2[u], b[0], b[1]);
          mma(o[u][2 * c + 1], lo2[u], b[2], b[3]);
        }
      }
    }
    const bool last = at.tile == at.tiles - 1;
    if (last || i == count - 1) {
      const bool whole = last && first_tile == 0;
#pragma unroll
      for (int u = 0; u < kTiles; ++u)
#pragma unroll
        for (int w = 0; w < (MT == 0 ? 1 : 2); ++w) {
          float sum = l[u][w];
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          const int h = u * 16 + g + w * 8;
          if (h >= heads) continue;
          const int64_t head = (whole ? (int64_t)at.b : (int64_t)r + at.b) * a.heads + h0 + h;
          const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            const int d = n * 8 + t * 2;
            if (d >= D) continue;
            float x = o[u][n][2 * w], y = o[u][n][2 * w + 1];
            if constexpr (MT == 0) {
              x += o[u][n][2];
              y += o[u][n][3];
            }
            if (whole) {
              *reinterpret_cast<uint32_t*>(static_cast<char*>(a.out) + (head * D + d) * 2) = pack_bf16x2(x * inv, y * inv);
            } else {
              *reinterpret_cast<float2*>(a.part_o + head * D + d) = make_float2(x, y);
            }
          }
          if (t == 0) {
            if (!whole) {
              a.part_ml[head] = make_float2(m[u][w], sum);
            } else if (a.lse != nullptr) {
              a.lse[head] = sum > 0.0f ? (m[u][w] + log2f(sum)) * kLn2 : -INFINITY;
            }
          }
        }
      fresh = true;
    }
    if (i + 1 < count) at.next(a);
  }
}

// Joins the parts of the sequences that more than one range covers, and
// answers for those without a position. Many parts of a head are shared by up
// to eight warps, whose sums are joined in shared memory.
template <typename ET>
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendArgs a) {
  __shared__ int s_total[8], s_before[8];
  __shared__ float s_o[8][MOE_ATTENTION_MAX_DIM];
  __shared__ float2 s_ml[8];
  const int lane = lane_id(), warp = threadIdx.x / kWarp, b = blockIdx.x;
  // The lengths are no output of the kernel before, which starts this one early.
  int total = 0, before = 0;  // tiles of all sequences, and of those in front of b
  for (int i = threadIdx.x; i < a.seqs; i += blockDim.x) {
    const int t = tiles_of(a, i);
    total += t;
    if (i < b) before += t;
  }
#pragma unroll
  for (int d = 1; d < kWarp; d <<= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, d);
    before += __shfl_xor_sync(0xffffffffu, before, d);
  }
  if (lane == 0) {
    s_total[warp] = total;
    s_before[warp] = before;
  }
  __syncthreads();
  total = before = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    total += s_total[w];
    before += s_before[w];
  }
  const int tiles = tiles_of(a, b), D = a.D;
  int r0 = 0, parts = 0;
  if (tiles > 0) {
    const int ranges = ranges_of(a, total);
    r0 = range_at(before, ranges, total);
    parts = range_at(before + tiles - 1, ranges, total) - r0 + 1;
  }
  await_previous_kernel();
  if (parts == 1) return;
  const int split = parts <= 4 ? 1 : parts <= 8 ? 2 : parts <= 16 ? 4 : 8;  // warps of a head
  const int at_once = 8 / split, sub = warp % split;
  for (int h0 = blockIdx.y * at_once; h0 < a.heads; h0 += gridDim.y * at_once) {
    const int h = h0 + warp / split;
    float m = -INFINITY, sum = 0.0f, o[MOE_ATTENTION_MAX_DIM / kWarp];
#pragma unroll
    for (int j = 0; j < MOE_ATTENTION_MAX_DIM / kWarp; ++j) o[j] = 0.0f;
    if (h < a.heads) {
      const int64_t first = (int64_t)(r0 + b) * a.heads + h;  // of part 0; the next is a.heads further
      for (int i0 = sub; i0 < parts; i0 += split * kWarp) {  // 32 of this warp's parts at a time
        const int mine = i0 + lane * split, n = min(kWarp, (parts - i0 + split - 1) / split);
        const float2 ml = mine < parts ? a.part_ml[first + (int64_t)mine * a.heads] : make_float2(-INFINITY, 0.0f);
        float top = ml.x;
#pragma unroll
        for (int d = 1; d < kWarp; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float now = fmaxf(m, top), base = now == -INFINITY ? 0.0f : now;
        const float keep = exp2f(m - base), weight = exp2f(ml.x - base);
        m = now;
        float all = ml.y * weight;
#pragma unroll
        for (int d = 1; d < kWarp; d <<= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
        sum = sum * keep + all;
#pragma unroll
        for (int j = 0; j < MOE_ATTENTION_MAX_DIM / kWarp; ++j) o[j] *= keep;
        const float* rows = a.part_o + (first + (int64_t)i0 * a.heads) * D;
        const int64_t step = (int64_t)split * a.heads * D;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
          const float w = __shfl_sync(0xffffffffu, weight, i);
#pragma unroll
          for (int j = 0; j < MOE_ATTENTION_MAX_DIM / kWarp; ++j)
            if (j * kWarp + lane < D) o[j] = fmaf(w, rows[i * step + j * kWarp + lane], o[j]);
        }
      }
    }
    if (split > 1) {
      __syncthreads();
      if (lane == 0) s_ml[warp] = make_float2(m, sum);
#pragma unroll
      for (int j = 0; j < MOE_ATTENTION_MAX_DIM / kWarp; ++j) s_o[warp][j * kWarp + lane] = o[j];
      __syncthreads();
      if (sub != 0) continue;
      float top = -INFINITY;
      for (int w = 0; w < split; ++w) top = fmaxf(top, s_ml[warp + w].x);
      m = top;
      sum = 0.0f;
#pragma unroll
      for (int j = 0; j < MOE_ATTENTION_MAX_DIM / kWarp; ++j) o[j] = 0.0f;
      const float base = top == -INFINITY ? 0.0f : top;
      for (int w = 0; w < split; ++w) {
        const float2 ml = s_ml[warp + w];
        const float weight = exp2f(ml.x - base);
        sum += ml.y * weight;
#pragma unroll
        for (int j = 0; j < MOE_ATTENTION_MAX_DIM / kWarp; ++j) o[j] = fmaf(weight, s_o[warp + w][j * kWarp + lane], o[j]);
      }
    }
    if (h >= a.heads) continue;
    const int64_t head = (int64_t)b * a.heads + h;
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int j = 0; j < MOE_ATTENTION_MAX_DIM / kWarp; ++j) {
      const int d = j * kWarp + lane;
      if (d >= D) continue;
      if constexpr (sizeof(ET) == 4) {
        static_cast<float*>(a.out)[head * D + d] = o[j] * inv;
      } else {
        static_cast<__nv_bfloat16*>(a.out)[head * D + d] = __float2bfloat16_rn(o[j] * inv);
      }
    }
    if (lane == 0 && a.lse != nullptr) a.lse[head] = sum > 0.0f ? (m + log2f(sum)) * kLn2 : -INFINITY;
  }
}

// Ranges of the line for a kernel of `warps` warps an SM that takes kHeads query heads at a time.
void cut(AttendArgs& a, int heads_at_once, int warps) {
  a.parts = (a.group + heads_at_once - 1) / heads_at_once;
  const int64_t r = (int64_t)num_sms() * warps / ((int64_t)a.kv_heads * a.parts);
  a.ranges = (int32_t)(r < 1 ? 1 : r);
}
unsigned ctas_of(const AttendArgs& a, int warps) {
  return (unsigned)(((int64_t)a.ranges * a.kv_heads * a.parts + warps - 1) / warps);
}

template <typename ET, int GM, int NC> int launch_rows(AttendArgs& a, cudaStream_t s) {
  static std::atomic<bool> raised[kSmemDevices];
  auto k = attend_rows_kernel<ET, GM, NC>;
  if (!allow_smem(k, raised)) return MOE_ERR_CUDA;
  cut(a, GM, kSmWarps);
  const int quads = (((a.D + 3) / 4) + 3) / 4;
  const int pitch = (quads * 4 + ((quads & 1) ? 0 : 4)) * 4;
  const size_t smem = (size_t)kSmWarps * (2 * 8 * pitch + GM * pitch + GM * 8) * 4;
  launch(k, dim3(ctas_of(a, kSmWarps)), dim3(kSmWarps * kWarp), smem, s, a);
  return check_launch();
}
template <typename ET, int GM> int launch_rows_dim(AttendArgs& a, cudaStream_t s) {
  return a.D <= 128 ? launch_rows<ET, GM, 1>(a, s) : launch_rows<ET, GM, 2>(a, s);
}
template <int DP, int MT> int launch_mma(AttendArgs& a, cudaStream_t s) {
  using S = Mma<DP, MT>;
  static std::atomic<bool> raised[kSmemDevices];
  auto k = attend_mma_kernel<DP, MT>;
  if (!allow_smem(k, raised)) return MOE_ERR_CUDA;
  cut(a, S::kHeads, S::kWarps);
  launch(k, dim3(ctas_of(a, S::kWarps)), dim3(S::kWarps * kWarp), S::kSmem, s, a);
  return check_launch();
}
template <int DP> int launch_mma_heads(AttendArgs& a, cudaStream_t s) {
  if (a.group <= 8) return launch_mma<DP, 0>(a, s);
  if constexpr (DP < 256)  // two tiles of heads at once: the registers hold them up to 128 elements
    if (a.group > 16) return launch_mma<DP, 2>(a, s);
  return launch_mma<DP, 1>(a, s);
}
template <typename ET> int run_attend(AttendArgs& a, cudaStream_t s) {
  int rc;
  // Rows of 16-byte pieces on 16 bytes (and query rows and outputs on 4) go to the tensor cores.
  const int64_t pieces = a.page_stride | a.token_stride | a.head_stride | (int64_t)(reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) |
                         (int64_t)(reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new)) | a.kn_row | a.kn_head |
                         a.vn_row | a.vn_head | a.D * (int64_t)sizeof(ET);
  const int64_t pairs = a.q_row | a.q_head | (int64_t)(reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.out));
  if (sizeof(ET) == 2 && pieces % 16 == 0 && pairs % 4 == 0) {
    rc = a.D <= 64 ? launch_mma_heads<64>(a, s) : a.D <= 128 ? launch_mma_heads<128>(a, s) : launch_mma_heads<256>(a, s);
  } else {
    rc = a.group == 1 ? launch_rows_dim<ET, 1>(a, s)
         : a.group == 2 ? launch_rows_dim<ET, 2>(a, s)
         : a.group <= 4 ? launch_rows_dim<ET, 4>(a, s)
                        : launch_rows_dim<ET, 8>(a, s);
  }
  if (rc != MOE_OK) return rc;
  int y = (int)(4 * (int64_t)num_sms() / a.seqs);
  y = y < 1 ? 1 : (y > a.heads ? a.heads : y);
  launch(attend_join_kernel<ET>, dim3((unsigned)a.seqs, (unsigned)y), dim3(256), 0, s, a);
  return check_launch();
}

int64_t slots_of(int64_t seqs, int32_t kv_heads) {
  const int64_t r = (int64_t)num_sms() * kSmWarps / kv_heads;
  return (r < 1 ? 1 : r) + seqs;
}

bool heads_ok(const moe_heads* h) { return h->row_stride >= 0 && h->head_stride >= 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_attention_decode_workspace_size(int64_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                                      int32_t head_dim) {
  if (num_seqs < 0 || num_seqs > MOE_CACHE_MAX_ROWS || num_kv_heads < 1 || num_heads < 1 || num_heads % num_kv_heads ||
      head_dim < 1 || head_dim > MOE_ATTENTION_MAX_DIM)
    return 0;
  const int64_t rows = slots_of(num_seqs, num_kv_heads) * num_heads;
  return (size_t)(rows * head_dim * 4 + 15) / 16 * 16 + (size_t)rows * 8;
}

extern "C" int moe_attention_decode(const moe_kv_cache* cache, const moe_heads* q, int32_t num_heads,
                                    const int32_t* page_table, int64_t table_stride, int64_t table_width,
                                    const int32_t* lengths, int64_t num_seqs, const moe_heads* k_new,
                                    const moe_heads* v_new, float scale, int64_t window, void* out, float* lse,
                                    void* workspace, size_t workspace_bytes, int32_t* d_status, moe_stream_t stream) {
  if (cache == nullptr || q == nullptr || (k_new == nullptr) != (v_new == nullptr)) return MOE_ERR_INVALID_ARG;
  const int eb = dtype_bytes(cache->dtype);
  if (eb == 0) return MOE_ERR_UNSUPPORTED;
  if (num_seqs < 0 || num_heads < 1 || cache->num_kv_heads < 1 || num_heads % cache->num_kv_heads ||
      cache->head_dim < 1 || cache->page_size < 1 || cache->num_pages < 0 || cache->page_stride < 0 ||
      cache->token_stride < 0 || cache->head_stride < 0 || table_width < 0 || window < 0 || !(fabsf(scale) < INFINITY))
    return MOE_ERR_INVALID_ARG;
  if ((num_seqs > 1 && table_stride < table_width) || !heads_ok(q) || (k_new != nullptr && !(heads_ok(k_new) && heads_ok(v_new))))
    return MOE_ERR_INVALID_ARG;
  if (cache->head_dim > MOE_ATTENTION_MAX_DIM || num_seqs > MOE_CACHE_MAX_ROWS || cache->num_pages > INT32_MAX ||
      table_width > INT32_MAX || table_width * cache->page_size > INT32_MAX - kTile ||
      num_seqs * (table_width * cache->page_size) >= (int64_t)1 << 34)
    return MOE_ERR_UNSUPPORTED;
  if (num_seqs == 0) return MOE_OK;
  if ((cache->num_pages > 0 && (cache->k == nullptr || cache->v == nullptr)) || q->data == nullptr ||
      (table_width > 0 && page_table == nullptr) || lengths == nullptr || out == nullptr || workspace == nullptr ||
      (k_new != nullptr && (k_new->data == nullptr || v_new->data == nullptr)))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_attention_decode_workspace_size(num_seqs, num_heads, cache->num_kv_heads, cache->head_dim))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(cache->k, eb) || !aligned(cache->v, eb) || !aligned(q->data, eb) || !aligned(out, eb) || !aligned(page_table, 4) ||
      !aligned(lengths, 4) || !aligned(lse, 4) || !aligned(workspace, 16) || !aligned(d_status, 4) ||
      (k_new != nullptr && !(aligned(k_new->data, eb) && aligned(v_new->data, eb))))
    return MOE_ERR_UNSUPPORTED;
  AttendArgs a = {};
  a.k = static_cast<char*>(cache->k);
  a.v = static_cast<char*>(cache->v);
  a.page_stride = cache->page_stride * eb;
  a.token_stride = cache->token_stride * eb;
  a.head_stride = cache->head_stride * eb;
  a.q = static_cast<const char*>(q->data);
  a.q_row = q->row_stride * eb;
  a.q_head = q->head_stride * eb;
  if (k_new != nullptr) {
    a.k_new = static_cast<const char*>(k_new->data);
    a.v_new = static_cast<const char*>(v_new->data);
    a.kn_row = k_new->row_stride * eb;
    a.kn_head = k_new->head_stride * eb;
    a.vn_row = v_new->row_stride * eb;
    a.vn_head = v_new->head_stride * eb;
  }
  a.table = page_table;
  a.table_stride = table_stride;
  a.lengths = lengths;
  a.out = out;
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  const int64_t rows = slots_of(num_seqs, cache->num_kv_heads) * num_heads;
  a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + (rows * cache->head_dim * 4 + 15) / 16 * 16);
  a.status = d_status;
  a.page = Divisor((uint32_t)cache->page_size);
  a.num_pages = cache->num_pages;
  a.window = window;
  a.seqs = (int32_t)num_seqs;
  a.width = (int32_t)table_width;
  a.heads = num_heads;
  a.kv_heads = cache->num_kv_heads;
  a.group = num_heads / cache->num_kv_heads;
  a.D = cache->head_dim;
  a.max_tokens = (int32_t)(table_width * cache->page_size);
  a.scale = scale * kLog2e;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return eb == 4 ? run_attend<float>(a, s) : run_attend<__nv_bfloat16>(a, s);
}
