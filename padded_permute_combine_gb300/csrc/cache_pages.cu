// The pages of a key-value cache: writing prompts into them, the page table of
// the next step (rows that go on, fork or end), compaction of the pool, and the
// copies that both ask for.
//
// A pool keeps no counts: a page is in use when a row of the table names it.
// Both table kernels run as one cluster of eight CTAs. Its shared memory holds a
// bit for every page of the pool, in eight slices; all CTAs set the bits of the
// rows' pages in it, and after the cluster's barrier each counts its own slice,
// so the i-th free page is known without a second launch, and without a word of
// workspace to clear. The barriers are the hardware's, of one cluster: its CTAs
// run together or not at all.
#include <cooperative_groups.h>

#include <atomic>

#include "block_common.h"
#include "common.cuh"
#include "moe_decode.h"

namespace moe {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------ write

struct WriteArgs {
  char* k;
  char* v;
  int64_t page_stride, token_stride, head_stride;  // bytes
  const char* k_new;
  const char* v_new;
  int64_t k_row, k_head, v_row, v_head;
  const int32_t* offsets;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lengths;
  int32_t* status;
  int64_t tokens, num_pages, width;
  int32_t seqs, kv_heads, page, row_bytes;
};

// A warp takes a token: all heads of its key, then of its value.
template <int VB>
__global__ void __launch_bounds__(256) cache_write_kernel(const WriteArgs a) {
  using V = typename Vec<VB>::T;
  await_previous_kernel();
  const int lane = lane_id(), warps = blockDim.x / kWarp;
  const int per_row = a.row_bytes / VB, per_token = per_row * a.kv_heads;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= a.seqs; i += blockDim.x) {
      const int64_t from = a.offsets[i], to = i < a.seqs ? a.offsets[i + 1] : a.tokens;
      if (from < 0 || from > to || (i == 0 && from != 0)) flag_status(a.status, MOE_STATUS_BAD_BINS);
    }
  for (int64_t t = (int64_t)blockIdx.x * warps + threadIdx.x / kWarp; t < a.tokens; t += (int64_t)gridDim.x * warps) {
    // The last sequence that begins at or before t, 32 ways at a time.
    int lo = 0, n = a.seqs + 1;  // entries lo .. lo + n - 1 of offsets may be it
    while (n > 1) {
      const int step = (n + kWarp - 1) / kWarp, i = lane * step;
      const bool le = i < n && a.offsets[lo + i] <= t;
      const unsigned hit = __ballot_sync(0xffffffffu, le);
      if (hit == 0) {
        n = 0;
        break;
      }
      const int j = (kWarp - 1 - __clz(hit)) * step;
      lo += j;
      n = min(step, n - j);
    }
    if (n == 0 || lo >= a.seqs) {
      if (n == 0 && lane == 0) flag_status(a.status, MOE_STATUS_BAD_BINS);
      continue;  // behind the last sequence
    }
    const int64_t end = a.offsets[lo + 1];
    if (a.offsets[lo] > t || end <= t || end > a.tokens || a.offsets[lo] < 0) {
      if (lane == 0) flag_status(a.status, MOE_STATUS_BAD_BINS);
      continue;
    }
    const int64_t pos = a.lengths[lo] - (end - t);
    const int64_t entry = pos / a.page;
    int page = -1;
    if (pos >= 0 && entry < a.width) page = a.table[lo * a.table_stride + entry];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) flag_status(a.status, MOE_STATUS_BAD_INDEX);
      continue;
    }
    const int64_t to = page * a.page_stride + (pos - entry * a.page) * a.token_stride;
    for (int i = lane; i < per_token; i += kWarp) {
      const int h = i / per_row, c = i - h * per_row;
      const int64_t dst = to + h * a.head_stride + (int64_t)c * VB;
      const V k = ld_stream(reinterpret_cast<const V*>(a.k_new + t * a.k_row + h * a.k_head + (int64_t)c * VB));
      const V v = ld_stream(reinterpret_cast<const V*>(a.v_new + t * a.v_row + h * a.v_head + (int64_t)c * VB));
      *reinterpret_cast<V*>(a.k + dst) = k;
      *reinterpret_cast<V*>(a.v + dst) = v;
    }
  }
}

// ------------------------------------------------------------------ tables

constexpr int kCtas = 8, kThreads = 1024, kWarps = kThreads / kWarp;

struct TableArgs {
  const int32_t* table;
  int64_t table_stride, width;
  const int32_t* lengths;
  const int32_t* parents;  // nullptr in compaction: every row is its own
  int32_t* new_table;
  int64_t new_width;
  int32_t* new_lengths;
  int32_t* src;
  int32_t* dst;
  int32_t* count;
  int32_t* status;
  int64_t seqs, rows, num_pages, grow, page;
  int32_t words_shift;  // log2 of the words of a slice
  int32_t hash_bits;
};

// What a row goes on from.
struct Parent {
  int row;      // -1: none
  int length;   // tokens
  int held;     // pages
};
__device__ __forceinline__ Parent parent_of(const TableArgs& a, int64_t r, bool flag) {
  Parent p = {(int)r, 0, 0};
  if (a.parents != nullptr) {
    p.row = a.parents[r];
    if (p.row < -1 || p.row >= a.seqs) {
      if (flag) flag_status(a.status, MOE_STATUS_BAD_INDEX);
      p.row = -1;
    }
  }
  if (p.row < 0) return p;
  const int64_t n = a.lengths[p.row], most = a.width * a.page;
  if (flag && (n < 0 || n > most)) flag_status(a.status, MOE_STATUS_BAD_INDEX);
  p.length = (int)(n < 0 ? 0 : (n > most ? most : n));
  p.held = (int)((p.length + a.page - 1) / a.page);
  return p;
}
__device__ __forceinline__ int page_of(const TableArgs& a, int row, int64_t j) {
  const int id = a.table[row * a.table_stride + j];
  return id >= 0 && id < a.num_pages ? id : -1;
}

// Sum over the CTA, and in `before` over the threads in front.
__device__ __forceinline__ int cta_prefix(int v, int* s_warp, int& before) {
  const int lane = lane_id(), warp = threadIdx.x / kWarp;
  int x = v;
#pragma unroll
  for (int d = 1; d < kWarp; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += o;
  }
  __syncthreads();
  if (lane == kWarp - 1) s_warp[warp] = x;
  __syncthreads();
  int y = s_warp[lane];  // kWarps == 32
#pragma unroll
  for (int d = 1; d < kWarp; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) y += o;
  }
  const int total = __shfl_sync(0xffffffffu, y, kWarps - 1);
  const int front = __shfl_sync(0xffffffffu, y, warp == 0 ? 0 : warp - 1);
  before = (warp == 0 ? 0 : front) + x - v;
  return total;
}

// Copies the rows' pages into the new table, with -1 behind them, and sets
// their bits. Rows go round over the cluster's CTAs, several warps to a row.
__device__ __forceinline__ void mark_rows(cg::cluster_group& cluster, const TableArgs& a, unsigned* bits) {
  const int rank = cluster.block_rank();
  const int64_t total = a.rows * a.new_width;
  // One entry a thread, in the table's order, so that few and many rows go alike.
  for (int64_t i = (int64_t)rank * kThreads + threadIdx.x; i < total; i += (int64_t)kCtas * kThreads) {
    const int64_t r = i / a.new_width, j = i - r * a.new_width;
    const Parent p = parent_of(a, r, false);
    int id = -1;
    if (j < p.held) {
      id = page_of(a, p.row, j);
      if (id < 0) {
        flag_status(a.status, MOE_STATUS_BAD_INDEX);
      } else {
        const int w = id >> 5;
        atomicOr(cluster.map_shared_rank(bits, w >> a.words_shift) + (w & ((1 << a.words_shift) - 1)), 1u << (id & 31));
      }
    }
    a.new_table[i] = id;
  }
}
// The bits of word w of this CTA's slice that are pages of the pool.
__device__ __forceinline__ unsigned pool_mask(const TableArgs& a, int rank, int w) {
  const int64_t first = (((int64_t)rank << a.words_shift) + w) * 32, n = a.num_pages - first;
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1) cache_fork_kernel(const TableArgs a) {
  extern __shared__ unsigned smem[];
  __shared__ int s_warp[kWarps], s_totals[kCtas];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), words = 1 << a.words_shift, R = (int)a.rows;
  unsigned* bits = smem;
  int* start = reinterpret_cast<int*>(smem + words);  // [R]: requests of the rows in front
  int* last = start + R;                              // [R]: page that is copied, or -1
  int* keys = last + R;                               // hash of the last pages that are not full
  int* vals = keys + (1 << a.hash_bits);              // the first row that holds one
  await_previous_kernel();
  for (int w = threadIdx.x; w < words; w += kThreads) bits[w] = 0;
  for (int i = threadIdx.x; i < 1 << a.hash_bits; i += kThreads) {
    keys[i] = -1;
    vals[i] = INT32_MAX;
  }
  cluster.sync();
  mark_rows(cluster, a, bits);
  // Every CTA knows all rows' requests.
  const unsigned mask = (1u << a.hash_bits) - 1;
  for (int r = threadIdx.x; r < R; r += kThreads) {
    const Parent p = parent_of(a, r, rank == 0);
    int id = -1;
    if (a.grow > 0 && p.row >= 0 && p.length % a.page != 0) {
      id = page_of(a, p.row, p.held - 1);
      if (id >= 0) {
        unsigned at = (unsigned)id * 2654435761u >> (32 - a.hash_bits);
        for (unsigned i = 0; i <= mask; ++i, at = (at + 1) & mask) {  // twice as many places as rows
          const int old = atomicCAS(&keys[at], -1, id);
          if (old == -1 || old == id) {
            atomicMin(&vals[at], r);
            break;
          }
        }
      }
    }
    last[r] = id;
  }
  __syncthreads();
  const int chunk = (R + kThreads - 1) / kThreads;
  int mine = 0;
  for (int r = threadIdx.x * chunk; r < R && r < (int)(threadIdx.x + 1) * chunk; ++r) {
    const Parent p = parent_of(a, r, false);
    int need = 0;
    if (p.row >= 0) {
      const int64_t want = (p.length + a.grow + a.page - 1) / a.page, all = want < a.new_width ? want : a.new_width;
      need = all > p.held ? (int)all - p.held : 0;
      if (rank == 0 && want > a.new_width) flag_status(a.status, MOE_STATUS_NO_PAGES);
    }
    if (last[r] >= 0) {
      unsigned at = (unsigned)last[r] * 2654435761u >> (32 - a.hash_bits);
      for (unsigned i = 0; i <= mask && keys[at] != last[r]; ++i) at = (at + 1) & mask;
      if (vals[at] == r) last[r] = -1; else ++need;
    }
    start[r] = mine;
    mine += need;
  }
  int before;
  const int requests = cta_prefix(mine, s_warp, before);
  for (int r = threadIdx.x * chunk; r < R && r < (int)(threadIdx.x + 1) * chunk; ++r) start[r] += before;
  if (rank == 0) {
    for (int r = threadIdx.x; r < R; r += kThreads) {
      a.new_lengths[r] = parent_of(a, r, false).length;
      a.src[r] = a.dst[r] = -1;
    }
  }
  cluster.sync();  // all bits are set, and what the requests overwrite is written
  // Free pages in front of each word of the slice, and of the slice.
  const int per = (words + kThreads - 1) / kThreads;
  int free_here = 0;
  for (int w = threadIdx.x * per; w < words && w < (int)(threadIdx.x + 1) * per; ++w)
    free_here += __popc(~bits[w] & pool_mask(a, rank, w));
  const int slice = cta_prefix(free_here, s_warp, before);
  if (threadIdx.x < kCtas) cluster.map_shared_rank(s_totals, threadIdx.x)[rank] = slice;
  cluster.sync();
  int all_free = 0;
  for (int i = 0; i < kCtas; ++i) {
    if (i < rank) before += s_totals[i];
    all_free += s_totals[i];
  }
  if (rank == 0 && threadIdx.x == 0 && requests > all_free) flag_status(a.status, MOE_STATUS_NO_PAGES);
  // A warp hands out its words' pages, a word at a time, each lane one of its bits.
  const int lane = lane_id();
  for (int i = 0; i < per; ++i) {
    const int w = threadIdx.x * per + i;
    const unsigned own = w < words ? ~bits[w] & pool_mask(a, rank, w) : 0u;
    if (!__any_sync(0xffffffffu, own != 0 && before < requests)) break;  // a thread's later words begin no lower
    for (int k = 0; k < kWarp; ++k) {
      const unsigned free = __shfl_sync(0xffffffffu, own, k);
      const int base = __shfl_sync(0xffffffffu, before, k), word = __shfl_sync(0xffffffffu, w, k);
      const int q = base + __popc(free & lanemask_lt());
      if (base >= requests || !(free >> lane & 1) || q >= requests) continue;
      int lo = 0, hi = R;  // the last row whose requests begin at or before q
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start[mid] <= q) lo = mid; else hi = mid;
      }
      const Parent p = parent_of(a, lo, false);
      const int copied = last[lo] >= 0, id = (((rank << a.words_shift) + word) << 5) + lane;
      a.new_table[lo * a.new_width + p.held - copied + (q - start[lo])] = id;
      if (copied && q == start[lo]) {
        a.src[lo] = last[lo];
        a.dst[lo] = id;
      }
    }
    before += __popc(own);
  }
  // A copied page that none was free for: the row must not write the one that it shares.
  if (rank == 0)
    for (int r = threadIdx.x; r < R; r += kThreads)
      if (last[r] >= 0 && start[r] >= all_free) a.new_table[r * a.new_width + parent_of(a, r, false).held - 1] = -1;
  cluster.sync();  // no CTA leaves while others use its shared memory
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1) cache_compact_kernel(const TableArgs a) {
  extern __shared__ unsigned smem[];
  __shared__ int s_warp[kWarps], s_totals[kCtas];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), words = 1 << a.words_shift;
  unsigned* bits = smem;
  int* front = reinterpret_cast<int*>(smem + words);  // pages in use in front of each word
  await_previous_kernel();
  for (int w = threadIdx.x; w < words; w += kThreads) bits[w] = 0;
  cluster.sync();
  if (rank == 0)
    for (int r = threadIdx.x; r < a.rows; r += kThreads) (void)parent_of(a, r, true);
  mark_rows(cluster, a, bits);
  cluster.sync();
  const int per = (words + kThreads - 1) / kThreads;
  int used_here = 0;
  for (int w = threadIdx.x * per; w < words && w < (int)(threadIdx.x + 1) * per; ++w) used_here += __popc(bits[w]);
  int before;
  const int slice = cta_prefix(used_here, s_warp, before);
  if (threadIdx.x < kCtas) cluster.map_shared_rank(s_totals, threadIdx.x)[rank] = slice;
  cluster.sync();
  int live = 0;
  for (int i = 0; i < kCtas; ++i) {
    if (i < rank) before += s_totals[i];
    live += s_totals[i];
  }
  for (int w = threadIdx.x * per, x = before; w < words && w < (int)(threadIdx.x + 1) * per; ++w) {
    front[w] = x;
    x += __popc(bits[w]);
  }
  cluster.sync();
  // Pages in use in front of page number `id`.
  const auto used_before = [&](int id) {
    const int w = id >> 5, at = w & (words - 1), in = w >> a.words_shift;
    if (in >= kCtas) return live;
    return cluster.map_shared_rank(front, in)[at] + __popc(cluster.map_shared_rank(bits, in)[at] & ((1u << (id & 31)) - 1));
  };
  const int kept = used_before(live), moves = live - kept;  // in use below `live`; holes there = live - kept
  for (int w = threadIdx.x * per; w < words && w < (int)(threadIdx.x + 1) * per; ++w) {
    const int first = ((rank << a.words_shift) + w) << 5;
    unsigned used = bits[w];
    const unsigned low = first + 32 <= live ? 0xffffffffu : first >= live ? 0u : (1u << (live - first)) - 1;  // pages below `live`
    unsigned holes = ~used & low, movers = used & ~low;
    for (int x = first - front[w]; holes != 0; holes &= holes - 1) {  // holes in front of the word's first
      const int bit = __ffs(holes) - 1;
      a.dst[x + __popc(~used & ((1u << bit) - 1))] = first + bit;
    }
    for (; movers != 0; movers &= movers - 1) {
      const int bit = __ffs(movers) - 1;
      a.src[front[w] + __popc(used & ((1u << bit) - 1)) - kept] = first + bit;
    }
  }
  for (int64_t i = moves + (int64_t)rank * kThreads + threadIdx.x; i < a.num_pages / 2; i += kCtas * kThreads)
    a.src[i] = a.dst[i] = -1;
  if (rank == 0 && threadIdx.x == 0) *a.count = moves;
  cluster.sync();
  // Entries at or above `live` get their new numbers: each thread those that it wrote itself.
  for (int64_t i = (int64_t)rank * kThreads + threadIdx.x; i < a.rows * a.new_width; i += (int64_t)kCtas * kThreads) {
    const int id = a.new_table[i];
    if (id >= live) a.new_table[i] = __ldcg(a.dst + (used_before(id) - kept));
  }
  cluster.sync();
}

int words_shift_of(int64_t num_pages) {
  const int64_t words = (num_pages + 31) / 32;
  int s = 0;
  while (((int64_t)kCtas << s) < words) ++s;
  return s;
}

int launch_table(void (*k)(TableArgs), std::atomic<bool>* raised, const TableArgs& a, size_t smem, cudaStream_t s) {
  if (!allow_smem(k, raised)) return MOE_ERR_CUDA;
  launch(k, dim3(kCtas), dim3(kThreads), smem, s, a);
  return check_launch();
}

bool table_ok(int64_t table_stride, int64_t table_width, int64_t num_seqs, int32_t page_size, int64_t num_pages) {
  return num_seqs >= 0 && table_width >= 0 && page_size >= 1 && num_pages >= 0 && (num_seqs < 2 || table_stride >= table_width);
}
bool table_supported(int64_t table_width, int64_t num_seqs, int32_t page_size, int64_t num_pages) {
  return num_seqs <= MOE_CACHE_MAX_ROWS && num_pages <= MOE_CACHE_MAX_PAGES && table_width <= INT32_MAX &&
         table_width * page_size <= INT32_MAX;
}

// ------------------------------------------------------------------ copies

struct CopyArgs {
  moe_cache_pages caches[MOE_CACHE_MAX_CACHES];
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;
  int32_t* status;
  int64_t num_copies, num_pages;
};

constexpr int kCopyThreads = 256;
constexpr int64_t kPieceBytes = 16384;  // of a page, for a CTA at a time

// CTA (x, y): every gridDim.x-th pair in piece y of the caches' pages, counted over all caches.
__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(const __grid_constant__ CopyArgs a, int num_caches) {
  await_previous_kernel();
  int64_t n = a.num_copies;
  if (a.count != nullptr) {
    const int64_t c = *a.count;
    n = c < n ? (c < 0 ? 0 : c) : n;
  }
  int64_t y = blockIdx.y;
  int c = 0;
  for (; c < num_caches; ++c) {
    const int64_t pieces = (a.caches[c].page_bytes + kPieceBytes - 1) / kPieceBytes;
    if (y < pieces) break;
    y -= pieces;
  }
  if (c == num_caches) return;
  const int64_t from = y * kPieceBytes, left = a.caches[c].page_bytes - from;
  const int64_t bytes = left < kPieceBytes ? left : kPieceBytes;
  char* base = static_cast<char*>(a.caches[c].data) + from;
  const int64_t stride = a.caches[c].page_stride;
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const int s = a.src[i], d = a.dst[i];
    if (s < 0 || d < 0) continue;
    if (s >= a.num_pages || d >= a.num_pages) {
      if (threadIdx.x == 0) flag_status(a.status, MOE_STATUS_BAD_INDEX);
      continue;
    }
    const char* in = base + s * stride;
    char* out = base + d * stride;
    if (((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out) | (uintptr_t)bytes) & 15) == 0) {
      for (int64_t k = threadIdx.x; k < bytes / 16; k += kCopyThreads)
        reinterpret_cast<uint4*>(out)[k] = ld_stream(reinterpret_cast<const uint4*>(in) + k);
    } else {
      for (int64_t k = threadIdx.x; k < bytes; k += kCopyThreads) out[k] = in[k];
    }
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_cache_write(const moe_kv_cache* cache, const moe_heads* k, const moe_heads* v, int64_t num_tokens,
                               const int32_t* offsets, const int32_t* page_table, int64_t table_stride,
                               int64_t table_width, const int32_t* lengths, int64_t num_seqs, int32_t* d_status,
                               moe_stream_t stream) {
  if (cache == nullptr || k == nullptr || v == nullptr) return MOE_ERR_INVALID_ARG;
  const int eb = dtype_bytes(cache->dtype);
  if (eb == 0) return MOE_ERR_UNSUPPORTED;
  if (num_tokens < 0 || num_seqs < 0 || cache->num_kv_heads < 1 || cache->head_dim < 1 || cache->page_size < 1 ||
      cache->num_pages < 0 || cache->page_stride < 0 || cache->token_stride < 0 || cache->head_stride < 0 ||
      table_width < 0 || (num_seqs > 1 && table_stride < table_width) || k->row_stride < 0 || k->head_stride < 0 ||
      v->row_stride < 0 || v->head_stride < 0)
    return MOE_ERR_INVALID_ARG;
  if (cache->head_dim > (1 << 20) || (int64_t)cache->num_kv_heads * cache->head_dim > (1 << 26) || num_tokens > INT32_MAX ||
      num_seqs >= INT32_MAX || cache->num_pages > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (num_tokens == 0 || num_seqs == 0) return MOE_OK;
  if (k->data == nullptr || v->data == nullptr || offsets == nullptr || lengths == nullptr ||
      (table_width > 0 && page_table == nullptr) || (cache->num_pages > 0 && (cache->k == nullptr || cache->v == nullptr)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(cache->k, eb) || !aligned(cache->v, eb) || !aligned(k->data, eb) || !aligned(v->data, eb) || !aligned(offsets, 4) ||
      !aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(d_status, 4))
    return MOE_ERR_UNSUPPORTED;
  WriteArgs a = {};
  a.k = static_cast<char*>(cache->k);
  a.v = static_cast<char*>(cache->v);
  a.page_stride = cache->page_stride * eb;
  a.token_stride = cache->token_stride * eb;
  a.head_stride = cache->head_stride * eb;
  a.k_new = static_cast<const char*>(k->data);
  a.v_new = static_cast<const char*>(v->data);
  a.k_row = k->row_stride * eb;
  a.k_head = k->head_stride * eb;
  a.v_row = v->row_stride * eb;
  a.v_head = v->head_stride * eb;
  a.offsets = offsets;
  a.table = page_table;
  a.table_stride = table_stride;
  a.lengths = lengths;
  a.status = d_status;
  a.tokens = num_tokens;
  a.num_pages = cache->num_pages;
  a.width = table_width;
  a.seqs = (int32_t)num_seqs;
  a.kv_heads = cache->num_kv_heads;
  a.page = cache->page_size;
  a.row_bytes = cache->head_dim * eb;
  // Vectors as wide as every row's start and length allow.
  const int64_t all = a.row_bytes | a.page_stride | a.token_stride | a.head_stride | a.k_row | a.k_head | a.v_row | a.v_head |
                      (int64_t)(reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                                reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t ctas = (num_tokens + 7) / 8;
  const auto go = [&](auto kernel) { launch(kernel, dim3((unsigned)(ctas < 65535 ? ctas : 65535)), dim3(256), 0, s, a); };
  if (all % 16 == 0) go(cache_write_kernel<16>);
  else if (all % 8 == 0) go(cache_write_kernel<8>);
  else if (all % 4 == 0) go(cache_write_kernel<4>);
  else go(cache_write_kernel<2>);
  return check_launch();
}

extern "C" int moe_cache_fork(const int32_t* page_table, int64_t table_stride, int64_t table_width, const int32_t* lengths,
                              int64_t num_seqs, const int32_t* parents, int64_t num_rows, int32_t page_size,
                              int64_t num_pages, int64_t grow, int32_t* new_table, int64_t new_width,
                              int32_t* new_lengths, int32_t* src, int32_t* dst, int32_t* d_status,
                              moe_stream_t stream) {
  if (!table_ok(table_stride, table_width, num_seqs, page_size, num_pages) || num_rows < 0 || grow < 0 || new_width < 0)
    return MOE_ERR_INVALID_ARG;
  if (!table_supported(table_width, num_seqs, page_size, num_pages) || num_rows > MOE_CACHE_MAX_ROWS || new_width > INT32_MAX ||
      grow > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (new_width < table_width) return MOE_ERR_INVALID_ARG;
  if (num_rows == 0) return MOE_OK;
  if ((num_seqs > 0 && (lengths == nullptr || (table_width > 0 && page_table == nullptr))) || parents == nullptr ||
      (new_width > 0 && new_table == nullptr) || new_lengths == nullptr || src == nullptr || dst == nullptr)
    return MOE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)page_table, (const void*)lengths, (const void*)parents, (const void*)new_table,
                        (const void*)new_lengths, (const void*)src, (const void*)dst, (const void*)d_status})
    if (!aligned(p, 4)) return MOE_ERR_UNSUPPORTED;
  TableArgs a = {};
  a.table = page_table;
  a.table_stride = table_stride;
  a.width = table_width;
  a.lengths = lengths;
  a.parents = parents;
  a.new_table = new_table;
  a.new_width = new_width;
  a.new_lengths = new_lengths;
  a.src = src;
  a.dst = dst;
  a.status = d_status;
  a.seqs = num_seqs;
  a.rows = num_rows;
  a.num_pages = num_pages;
  a.grow = grow;
  a.page = page_size;
  a.words_shift = words_shift_of(num_pages);
  a.hash_bits = 1;
  while ((1 << a.hash_bits) < 2 * num_rows) ++a.hash_bits;
  const size_t smem = 4 * ((size_t)(1 << a.words_shift) + 2 * num_rows + 2 * ((size_t)1 << a.hash_bits));
  static std::atomic<bool> raised[kSmemDevices];
  return launch_table(cache_fork_kernel, raised, a, smem, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_cache_compact(const int32_t* page_table, int64_t table_stride, int64_t table_width,
                                 const int32_t* lengths, int64_t num_seqs, int32_t page_size, int64_t num_pages,
                                 int32_t* new_table, int32_t* src, int32_t* dst, int32_t* count, int32_t* d_status,
                                 moe_stream_t stream) {
  if (!table_ok(table_stride, table_width, num_seqs, page_size, num_pages)) return MOE_ERR_INVALID_ARG;
  if (!table_supported(table_width, num_seqs, page_size, num_pages)) return MOE_ERR_UNSUPPORTED;
  if ((num_seqs > 0 && (lengths == nullptr || (table_width > 0 && (page_table == nullptr || new_table == nullptr)))) ||
      (num_pages > 1 && (src == nullptr || dst == nullptr)) || count == nullptr)
    return MOE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)page_table, (const void*)lengths, (const void*)new_table, (const void*)src, (const void*)dst,
                        (const void*)count, (const void*)d_status})
    if (!aligned(p, 4)) return MOE_ERR_UNSUPPORTED;
  TableArgs a = {};
  a.table = page_table;
  a.table_stride = table_stride;
  a.width = table_width;
  a.lengths = lengths;
  a.new_table = new_table;
  a.new_width = table_width;
  a.src = src;
  a.dst = dst;
  a.count = count;
  a.status = d_status;
  a.seqs = a.rows = num_seqs;
  a.num_pages = num_pages;
  a.page = page_size;
  a.words_shift = words_shift_of(num_pages);
  static std::atomic<bool> raised[kSmemDevices];
  return launch_table(cache_compact_kernel, raised, a, (size_t)8 << a.words_shift, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_cache_copy(const moe_cache_pages* caches, int64_t num_caches, int64_t num_pages, const int32_t* src,
                              const int32_t* dst, int64_t num_copies, const int32_t* count, int32_t* d_status,
                              moe_stream_t stream) {
  if (num_caches < 0 || num_pages < 0 || num_copies < 0 || (num_caches > 0 && caches == nullptr)) return MOE_ERR_INVALID_ARG;
  if (num_caches > MOE_CACHE_MAX_CACHES || num_pages > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  CopyArgs a = {};
  int64_t pieces = 0;
  for (int64_t c = 0; c < num_caches; ++c) {
    if (caches[c].page_bytes < 0 || caches[c].page_stride < 0) return MOE_ERR_INVALID_ARG;
    if (num_pages > 1 && caches[c].page_stride < caches[c].page_bytes) return MOE_ERR_INVALID_ARG;
    if (num_pages > 0 && caches[c].page_bytes > 0 && caches[c].data == nullptr) return MOE_ERR_INVALID_ARG;
    a.caches[c] = caches[c];
    pieces += (caches[c].page_bytes + kPieceBytes - 1) / kPieceBytes;
  }
  if (pieces > 65535) return MOE_ERR_UNSUPPORTED;
  if (num_copies == 0 || pieces == 0 || num_pages == 0) return MOE_OK;
  if (src == nullptr || dst == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(count, 4) || !aligned(d_status, 4)) return MOE_ERR_UNSUPPORTED;
  a.src = src;
  a.dst = dst;
  a.count = count;
  a.status = d_status;
  a.num_copies = num_copies;
  a.num_pages = num_pages;
  int64_t x = ((int64_t)num_sms() * 8 + pieces - 1) / pieces;
  x = x < num_copies ? x : num_copies;
  launch(cache_copy_kernel, dim3((unsigned)x, (unsigned)pieces), dim3(kCopyThreads), 0, reinterpret_cast<cudaStream_t>(stream),
         a, (int)num_caches);
  return check_launch();
}
