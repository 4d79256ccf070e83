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
#include "attend.h"

namespace moe {
namespace {

// A lane's elements of a row of D: fours of them (QUADS, where D is a multiple
// of four), or every 32nd.
template <bool QUADS, int kLanes> struct RowPart {
  float v[kLanes];
  __device__ __forceinline__ static int place(int j) { return QUADS ? (j / 4 * kWarp + lane_id()) * 4 + j % 4 : j * kWarp + lane_id(); }
  __device__ __forceinline__ void load(const float* row, int D) {
    if constexpr (QUADS) {
#pragma unroll
      for (int j = 0; j < kLanes; j += 4) {
        const float4 x = place(j) < D ? *reinterpret_cast<const float4*>(row + place(j)) : make_float4(0, 0, 0, 0);
        v[j] = x.x;
        v[j + 1] = x.y;
        v[j + 2] = x.z;
        v[j + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kLanes; ++j) v[j] = place(j) < D ? row[place(j)] : 0.0f;
    }
  }
};

// Joins the parts of the sequences that more than one range covers, and
// answers for those without a position. Many parts of a head are shared by up
// to WARPS warps, whose sums are joined in shared memory. kLanes: elements of a
// row for a lane.
template <typename ET, bool QUADS, int kLanes, int WARPS>
__global__ void __launch_bounds__(WARPS * kWarp) attend_join_kernel(const AttendArgs a) {
  __shared__ int s_total[WARPS], s_before[WARPS];
  __shared__ float s_o[WARPS][kLanes * kWarp];
  __shared__ float2 s_ml[WARPS];
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
  for (int w = 0; w < WARPS; ++w) {
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
  int split = 1;  // warps of a head: two parts or so each
  while (split < WARPS && 2 * split < parts) split *= 2;
  const int at_once = WARPS / split, sub = warp % split;
  for (int h0 = blockIdx.y * at_once; h0 < a.heads; h0 += gridDim.y * at_once) {
    const int h = h0 + warp / split;
    using P = RowPart<QUADS, kLanes>;
    constexpr int kAhead = WARPS * kLanes > 128 ? 4 : 8;  // parts on their way together, as the registers allow
    float m = -INFINITY, sum = 0.0f, o[kLanes];
#pragma unroll
    for (int j = 0; j < kLanes; ++j) o[j] = 0.0f;
    if (h < a.heads) {
      const int64_t first = (int64_t)(r0 + b) * a.heads + h;  // of part 0; the next is a.heads further
      for (int i0 = sub; i0 < parts; i0 += split * kWarp) {  // 32 of this warp's parts at a time
        const int mine = i0 + lane * split, n = min(kWarp, (parts - i0 + split - 1) / split);
        const float* rows = a.part_o + (first + (int64_t)i0 * a.heads) * D;
        const int64_t step = (int64_t)split * a.heads * D;
        const float2 ml = mine < parts ? a.part_ml[first + (int64_t)mine * a.heads] : make_float2(-INFINITY, 0.0f);
        P next[kAhead];  // the first parts are on their way with the maxima and sums
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (i < n) next[i].load(rows + i * step, D);
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
        for (int j = 0; j < kLanes; ++j) o[j] *= keep;
        for (int i = 0; i < n; i += kAhead) {
          if (i > 0) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
              if (i + k < n) next[k].load(rows + (i + k) * step, D);
          }
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            if (i + k >= n) continue;
            const float w = __shfl_sync(0xffffffffu, weight, i + k);
#pragma unroll
            for (int j = 0; j < kLanes; ++j) o[j] = fmaf(w, next[k].v[j], o[j]);
          }
        }
      }
    }
    if (split > 1) {
      __syncthreads();
      if (lane == 0) s_ml[warp] = make_float2(m, sum);
#pragma unroll
      for (int j = 0; j < kLanes; ++j) s_o[warp][P::place(j)] = o[j];
      __syncthreads();
      if (sub != 0) continue;
      float top = -INFINITY;
      for (int w = 0; w < split; ++w) top = fmaxf(top, s_ml[warp + w].x);
      m = top;
      sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kLanes; ++j) o[j] = 0.0f;
      const float base = top == -INFINITY ? 0.0f : top;
      for (int w = 0; w < split; ++w) {
        const float2 ml = s_ml[warp + w];
        const float weight = exp2f(ml.x - base);
        sum += ml.y * weight;
#pragma unroll
        for (int j = 0; j < kLanes; ++j) o[j] = fmaf(weight, s_o[warp + w][P::place(j)], o[j]);
      }
    }
    if (h >= a.heads) continue;
    const int64_t head = (int64_t)b * a.heads + h;
    const float inv = share_of(sum);
#pragma unroll
    for (int j = 0; j < kLanes; ++j) {
      const int d = P::place(j);
      if (d >= D) continue;
      if constexpr (sizeof(ET) == 4) {
        static_cast<float*>(a.out)[head * D + d] = o[j] * inv;
      } else {
        static_cast<__nv_bfloat16*>(a.out)[head * D + d] = __float2bfloat16_rn(o[j] * inv);
      }
    }
    if (lane == 0 && a.lse != nullptr) a.lse[head] = log_sum_of(m, sum);
  }
}

template <typename ET, bool QUADS> int launch_join(const AttendArgs& a, cudaStream_t s) {
  // Where a head may have more than 64 parts, 32 warps share it (one sequence of 80000 tokens, six heads of 600
  // parts: 26 us in all with eight warps, 21 with 32; 9 sequences with some 33 parts: 1 us more).
  const int most = a.max_tokens / kTile < a.ranges ? a.max_tokens / kTile : a.ranges;
  const bool few = most / a.seqs > 64;
  int y = (int)(4 * (int64_t)num_sms() / a.seqs);
  y = y < 1 ? 1 : (y > a.heads ? a.heads : y);
  const auto go = [&](auto kernel, int warps) { launch(kernel, dim3((unsigned)a.seqs, (unsigned)y), dim3(warps * kWarp), 0, s, a); };
  if (a.D <= 128) {
    if (few) go(attend_join_kernel<ET, QUADS, 4, 32>, 32); else go(attend_join_kernel<ET, QUADS, 4, 8>, 8);
  } else {
    if (few) go(attend_join_kernel<ET, QUADS, 8, 32>, 32); else go(attend_join_kernel<ET, QUADS, 8, 8>, 8);
  }
  return check_launch();
}
template <typename ET> int run_attend(AttendArgs& a, cudaStream_t s) {
  int rc;
  // What all rows are aligned to and multiples of, and query rows and outputs.
  const int64_t pieces = a.page_stride | a.token_stride | a.head_stride | (int64_t)(reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) |
                         (int64_t)(reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new)) | a.kn_row | a.kn_head |
                         a.vn_row | a.vn_head | a.D * (int64_t)sizeof(ET);
  const int64_t pairs = a.q_row | a.q_head | (int64_t)(reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.out));
  if constexpr (sizeof(ET) == 2) {
    rc = pairs % 4 != 0 || pieces % 4 != 0 ? attend_mma_2(a, s) : pieces % 16 != 0 ? attend_mma_4(a, s) : attend_mma_16(a, s);
  } else {
    rc = attend_rows(a, pieces % 16 == 0, s);
  }
  if (rc != MOE_OK) return rc;
  return a.D % 4 == 0 ? launch_join<ET, true>(a, s) : launch_join<ET, false>(a, s);
}

int64_t slots_of(int64_t seqs, int32_t kv_heads) {
  const int64_t r = (int64_t)num_sms() * kMostWarps / kv_heads;
  return (r < 1 ? 1 : r) + seqs;
}

constexpr int32_t kMostHeads = 1 << 30;  // with the last CTA's share, or the last step over heads, within 31 bits

bool heads_ok(const moe_heads* h) { return h->row_stride >= 0 && h->head_stride >= 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_attention_decode_workspace_size(int64_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                                      int32_t head_dim) {
  if (num_seqs < 0 || num_seqs > MOE_CACHE_MAX_ROWS || num_kv_heads < 1 || num_heads < 1 || num_heads > kMostHeads || num_heads % num_kv_heads ||
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
  if (cache->head_dim > MOE_ATTENTION_MAX_DIM || num_heads > kMostHeads || num_seqs > MOE_CACHE_MAX_ROWS || cache->num_pages > INT32_MAX ||
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
  if (cache->num_pages == 0) a.k = a.v = static_cast<char*>(workspace);  // an address for the copies of nothing
  const int64_t rows = slots_of(num_seqs, cache->num_kv_heads) * num_heads;
  a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + (rows * cache->head_dim * 4 + 15) / 16 * 16);
  a.status = d_status;
  a.page = Divisor((uint32_t)cache->page_size);
  a.num_pages = cache->num_pages;
  a.window = window;
  a.seqs = (int32_t)num_seqs;
  a.heads = num_heads;
  a.kv_heads = cache->num_kv_heads;
  a.group = num_heads / cache->num_kv_heads;
  a.D = cache->head_dim;
  a.max_tokens = (int32_t)(table_width * cache->page_size);
  a.scale = scale * kLog2e;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return eb == 4 ? run_attend<float>(a, s) : run_attend<__nv_bfloat16>(a, s);
}
