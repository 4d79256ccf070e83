// The pages of a key-value cache: writing prompts into them, the page table of
// the next step (rows that go on, fork or end), compaction of the pool, and the
// copies that both ask for.
//
// A pool keeps no counts: a page is in use when a row of the table names it.
// Both table kernels run as one CTA or, for large tables and pools, as one
// cluster of eight. Their shared memory holds a bit for every page of the pool
// (a slice of it in each CTA); the rows' pages set theirs, and after a barrier
// each CTA counts its own slice, so the i-th free page is known without a second
// launch, and without a word of workspace to clear. The barriers are the
// hardware's, of one cluster: its CTAs run together or not at all.
#include <cooperative_groups.h>

#include <atomic>

#include "block_common.h"
#include "common.cuh"
#include "divisor.h"
#include "moe_decode.h"
#include "search.h"

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
  Divisor page, per_row, per_token;  // vectors of a head's row, and of all heads'
  int32_t seqs, together;  // together: tokens that a warp takes at a time
};

// Where token t goes: bytes from the cache's start, or -1.
__device__ __forceinline__ int64_t place_of(const WriteArgs& a, int64_t t) {
  const int lo = last_at_most(a.offsets, a.seqs + 1, t);  // the last sequence that begins at or before t, if any
  const int64_t from = a.offsets[lo];
  if (lo == a.seqs && from <= t) return -1;  // behind the last sequence
  const int64_t end = lo < a.seqs ? a.offsets[lo + 1] : 0;
  if (from > t || from < 0 || end <= t || end > a.tokens) {
    flag_status(a.status, MOE_STATUS_BAD_BINS);
    return -1;
  }
  const int64_t pos = a.lengths[lo] - (end - t);
  const int64_t entry = pos < 0 ? 0 : a.page.of((uint32_t)pos);  // lengths have 32 bits
  int page = -1;
  if (pos >= 0 && entry < a.width) page = a.table[lo * a.table_stride + entry];
  if (page < 0 || page >= a.num_pages) {
    flag_status(a.status, MOE_STATUS_BAD_INDEX);
    return -1;
  }
  return page * a.page_stride + (pos - entry * a.page.d) * a.token_stride;
}

// A warp takes a few tokens at a time: as many lanes find their places, then
// all lanes copy their heads' vectors, one token's after the other.
template <int VB>
__global__ void __launch_bounds__(256) cache_write_kernel(const WriteArgs a) {
  using V = typename Vec<VB>::T;
  constexpr int kBatchVecs = 4;
  await_previous_kernel();
  const int lane = lane_id(), warps = blockDim.x / kWarp;
  const int per_token = (int)a.per_token.d;
  if (blockIdx.x == 0)
    for (uint32_t i = threadIdx.x; i <= (uint32_t)a.seqs; i += blockDim.x) {  // seqs may be all that 31 bits hold
      const int64_t from = a.offsets[i], to = i < a.seqs ? a.offsets[i + 1] : a.tokens;
      if (from < 0 || from > to || (i == 0 && from != 0)) flag_status(a.status, MOE_STATUS_BAD_BINS);
    }
  for (int64_t t0 = ((int64_t)blockIdx.x * warps + threadIdx.x / kWarp) * a.together; t0 < a.tokens; t0 += (int64_t)gridDim.x * warps * a.together) {
    const int n = a.tokens - t0 < a.together ? (int)(a.tokens - t0) : a.together;
    const int64_t mine = lane < n ? place_of(a, t0 + lane) : -1;
    for (int i0 = lane; i0 - lane < n * per_token; i0 += kBatchVecs * kWarp) {  // some vectors on their way together
      V k[kBatchVecs], v[kBatchVecs];
      int64_t dst[kBatchVecs];
#pragma unroll
      for (int e = 0; e < kBatchVecs; ++e) {
        const int i = i0 + e * kWarp;
        const int token = i < n * per_token ? (int)a.per_token.of(i) : 0;
        const int64_t to = __shfl_sync(0xffffffffu, mine, token);
        dst[e] = -1;
        if (i >= n * per_token || to < 0) continue;
        const int j = i - token * per_token, h = (int)a.per_row.of(j), c = (j - h * (int)a.per_row.d) * VB;
        dst[e] = to + h * a.head_stride + c;
        k[e] = ld_stream(reinterpret_cast<const V*>(a.k_new + (t0 + token) * a.k_row + h * a.k_head + c));
        v[e] = ld_stream(reinterpret_cast<const V*>(a.v_new + (t0 + token) * a.v_row + h * a.v_head + c));
      }
#pragma unroll
      for (int e = 0; e < kBatchVecs; ++e) {
        if (dst[e] < 0) continue;
        *reinterpret_cast<V*>(a.k + dst[e]) = k[e];
        *reinterpret_cast<V*>(a.v + dst[e]) = v[e];
      }
    }
  }
}

// ------------------------------------------------------------------ tables

constexpr int kThreads = 1024, kWarps = kThreads / kWarp;

// The CTAs of a table kernel.
template <int CTAS> struct Group {
  __device__ __forceinline__ static int rank() { return (int)cg::this_cluster().block_rank(); }
  __device__ __forceinline__ static void sync() { cg::this_cluster().sync(); }
  template <typename T> __device__ __forceinline__ static T* map(T* p, int rank) { return cg::this_cluster().map_shared_rank(p, rank); }
};
template <> struct Group<1> {
  __device__ __forceinline__ static int rank() { return 0; }
  __device__ __forceinline__ static void sync() { __syncthreads(); }
  template <typename T> __device__ __forceinline__ static T* map(T* p, int) { return p; }
};
constexpr int kBatch = 4;  // entries of the table that a thread takes at a time

struct TableArgs {
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lengths;
  const int32_t* parents;  // nullptr in compaction: every row is its own
  int32_t* new_table;
  int32_t* new_lengths;
  int32_t* src;
  int32_t* dst;
  int32_t* count;
  int32_t* status;
  Divisor page, columns;  // columns: of the new table
  int32_t width, new_width, seqs, rows, num_pages;
  int64_t grow;
  int32_t words_shift;  // log2 of the words of a slice
  int32_t whole;        // whether every CTA has bits of the whole pool, CTAS slices
  int32_t whole_at;     // in words of the shared memory
  int32_t hash_bits;
};

// What a row goes on from.
struct Parent {
  int row;     // -1: none
  int length;  // tokens
  int held;    // pages
};
__device__ __forceinline__ Parent parent_of(const TableArgs& a, int r, bool flag) {
  Parent p = {r, 0, 0};
  if (a.parents != nullptr) {
    p.row = a.parents[r];
    if (p.row < -1 || p.row >= a.seqs) {
      if (flag) flag_status(a.status, MOE_STATUS_BAD_INDEX);
      p.row = -1;
    }
  }
  if (p.row < 0) return p;
  const int n = a.lengths[p.row], most = a.width * (int)a.page.d;
  if (flag && (n < 0 || n > most)) flag_status(a.status, MOE_STATUS_BAD_INDEX);
  p.length = n < 0 ? 0 : (n > most ? most : n);
  p.held = (int)a.page.of(p.length);
  p.held += p.held * (int)a.page.d < p.length;
  return p;
}
__device__ __forceinline__ int page_of(const TableArgs& a, int row, int j) {
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
// their bits. The entries go round over all threads in the table's order, some
// at a time so that their loads are on their way together. s_row, s_held:
// every row's parent and pages.
template <int CTAS> __device__ __forceinline__ void mark_rows(const TableArgs& a, unsigned* bits, unsigned* whole, const int* s_row, const int* s_held) {
  using G = Group<CTAS>;
  const int total = a.rows * a.new_width;  // below 2^31 by more than the steps: checked at the call
  for (int i0 = G::rank() * kThreads + (int)threadIdx.x; i0 < total; i0 += kBatch * CTAS * kThreads) {
    int id[kBatch];
    bool in[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int i = i0 + e * CTAS * kThreads;
      if (i >= total) break;
      const int r = (int)a.columns.of(i), j = i - r * a.new_width;
      in[e] = j < s_held[r];
      id[e] = in[e] ? a.table[s_row[r] * a.table_stride + j] : -1;
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int i = i0 + e * CTAS * kThreads;
      if (i >= total) break;
      if (id[e] >= 0 && id[e] < a.num_pages) {
        const int w = id[e] >> 5;
        unsigned* at = CTAS == 1 || a.whole ? whole + w : G::map(bits, w >> a.words_shift) + (w & ((1 << a.words_shift) - 1));
        atomicOr(at, 1u << (id[e] & 31));
      } else {
        if (in[e]) flag_status(a.status, MOE_STATUS_BAD_INDEX);
        id[e] = -1;
      }
      a.new_table[i] = id[e];
    }
  }
}
template <int CTAS> __device__ __forceinline__ void clear_marks(const TableArgs& a, unsigned* bits, unsigned* whole) {
  const int words = 1 << a.words_shift;
  for (int w = threadIdx.x; w < words; w += kThreads) bits[w] = 0;
  if (CTAS > 1 && a.whole)
    for (int w = threadIdx.x; w < words * CTAS; w += kThreads) whole[w] = 0;
}
// Behind a barrier: this CTA's slice of the bits.
template <int CTAS> __device__ __forceinline__ void join_marks(const TableArgs& a, unsigned* bits, unsigned* whole) {
  if (CTAS == 1 || !a.whole) return;
  const int words = 1 << a.words_shift, rank = Group<CTAS>::rank();
  for (int w = threadIdx.x; w < words; w += kThreads) {
    unsigned v = 0;
#pragma unroll
    for (int k = 0; k < CTAS; ++k) v |= Group<CTAS>::map(whole, k)[(rank << a.words_shift) + w];
    bits[w] = v;
  }
  __syncthreads();
}
// The bits of word w of this CTA's slice that are pages of the pool.
__device__ __forceinline__ unsigned pool_mask(const TableArgs& a, int rank, int w) {
  const int64_t first = (((int64_t)rank << a.words_shift) + w) * 32, n = a.num_pages - first;
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
}

template <int CTAS> __global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kThreads, 1) cache_fork_kernel(const TableArgs a) {
  using G = Group<CTAS>;
  extern __shared__ unsigned smem[];
  __shared__ int s_warp[kWarps], s_totals[CTAS];
  const int rank = G::rank(), words = 1 << a.words_shift, R = a.rows;
  unsigned* bits = smem;
  int* row = reinterpret_cast<int*>(smem + words);  // [R]: parents
  int* held = row + R;                              // [R]: pages
  int* start = held + R;                            // [R]: requests of the rows in front
  int* last = start + R;                            // [R]: page that is copied, or -1
  int* keys = last + R;                             // hash of the last pages that are not full; then the words' free pages
  int* vals = keys + (1 << a.hash_bits);            // the first row that holds one
  unsigned* whole = CTAS == 1 ? bits : smem + a.whole_at;
  clear_marks<CTAS>(a, bits, whole);
  for (int i = threadIdx.x; i < 1 << a.hash_bits; i += kThreads) {
    keys[i] = -1;
    vals[i] = INT32_MAX;
  }
  await_previous_kernel();
  // Every CTA knows all rows.
  for (int r = threadIdx.x; r < R; r += kThreads) {
    const Parent p = parent_of(a, r, rank == 0);
    row[r] = p.row;
    held[r] = p.held;
    start[r] = p.length;  // for now
    last[r] = a.grow > 0 && p.row >= 0 && p.held * (int)a.page.d != p.length ? page_of(a, p.row, p.held - 1) : -1;
    if (rank == 0) {
      a.new_lengths[r] = p.length;
      a.src[r] = a.dst[r] = -1;
    }
  }
  G::sync();
  mark_rows<CTAS>(a, bits, whole, row, held);
  const unsigned mask = (1u << a.hash_bits) - 1;
  for (int r = threadIdx.x; r < R; r += kThreads) {
    const int id = last[r];
    if (id < 0) continue;
    unsigned at = (unsigned)id * 2654435761u >> (32 - a.hash_bits);
    for (unsigned i = 0; i <= mask; ++i, at = (at + 1) & mask) {  // twice as many places as rows
      const int old = atomicCAS(&keys[at], -1, id);
      if (old == -1 || old == id) {
        atomicMin(&vals[at], r);
        break;
      }
    }
  }
  __syncthreads();
  const int chunk = (R + kThreads - 1) / kThreads;
  int mine = 0;
  for (int r = threadIdx.x * chunk; r < R && r < (int)(threadIdx.x + 1) * chunk; ++r) {
    int need = 0;
    if (row[r] >= 0) {
      const int64_t tokens = start[r] + a.grow;  // at most 2^32
      const int64_t want = tokens < INT32_MAX ? a.page.of((uint32_t)tokens) + (a.page.of((uint32_t)tokens) * a.page.d < tokens)
                                              : (tokens + a.page.d - 1) / a.page.d;
      const int all = (int)(want < a.new_width ? want : a.new_width);
      need = all > held[r] ? all - held[r] : 0;
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
  G::sync();  // all bits are set, and what the requests overwrite is written
  join_marks<CTAS>(a, bits, whole);
  // Free pages in front of each word of the slice.
  int* front = keys;  // [words]: the hash is done with
  const int per = (words + kThreads - 1) / kThreads;
  int free_here = 0;
  for (int w = threadIdx.x * per; w < words && w < (int)(threadIdx.x + 1) * per; ++w)
    free_here += __popc(~bits[w] & pool_mask(a, rank, w));
  const int slice = cta_prefix(free_here, s_warp, before);
  if (threadIdx.x < CTAS) G::map(s_totals, threadIdx.x)[rank] = slice;
  G::sync();
  int all_free = 0;
  for (int i = 0; i < CTAS; ++i) {
    if (i < rank) before += s_totals[i];
    all_free += s_totals[i];
  }
  if (rank == 0 && threadIdx.x == 0 && requests > all_free) flag_status(a.status, MOE_STATUS_NO_PAGES);
  for (int w = threadIdx.x * per; w < words && w < (int)(threadIdx.x + 1) * per; ++w) {
    front[w] = before;
    before += __popc(~bits[w] & pool_mask(a, rank, w));
  }
  __syncthreads();
  // A warp hands out a word's pages, each lane one of its bits.
  const int lane = lane_id();
  for (int w = threadIdx.x / kWarp; w < words; w += kWarps) {
    if (front[w] >= requests) break;  // and neither are the later ones asked for
    const unsigned free = ~bits[w] & pool_mask(a, rank, w);
    const int q = front[w] + __popc(free & lanemask_lt());
    if (!(free >> lane & 1) || q >= requests) continue;
    int lo = 0, hi = R;  // the last row whose requests begin at or before q
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (start[mid] <= q) lo = mid; else hi = mid;
    }
    const int copied = last[lo] >= 0, id = (((rank << a.words_shift) + w) << 5) + lane;
    a.new_table[(int64_t)lo * a.new_width + held[lo] - copied + (q - start[lo])] = id;
    if (copied && q == start[lo]) {
      a.src[lo] = last[lo];
      a.dst[lo] = id;
    }
  }
  // A copied page that none was free for: the row must not write the one that it shares.
  if (rank == 0)
    for (int r = threadIdx.x; r < R; r += kThreads)
      if (last[r] >= 0 && start[r] >= all_free) a.new_table[(int64_t)r * a.new_width + held[r] - 1] = -1;
  // Nothing of another CTA is used behind the last barrier: none has to stay.
}

template <int CTAS> __global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kThreads, 1) cache_compact_kernel(const TableArgs a) {
  using G = Group<CTAS>;
  extern __shared__ unsigned smem[];
  __shared__ int s_warp[kWarps], s_totals[CTAS];
  const int rank = G::rank(), words = 1 << a.words_shift;
  unsigned* bits = smem;
  int* front = reinterpret_cast<int*>(smem + words);  // pages in use in front of each word
  int* row = front + words;                           // [rows]
  int* held = row + a.rows;                           // [rows]: pages
  unsigned* whole = CTAS == 1 ? bits : smem + a.whole_at;
  clear_marks<CTAS>(a, bits, whole);
  await_previous_kernel();
  for (int r = threadIdx.x; r < a.rows; r += kThreads) {
    row[r] = r;
    held[r] = parent_of(a, r, rank == 0).held;
  }
  G::sync();
  mark_rows<CTAS>(a, bits, whole, row, held);
  G::sync();
  join_marks<CTAS>(a, bits, whole);
  const int per = (words + kThreads - 1) / kThreads;
  int used_here = 0;
  for (int w = threadIdx.x * per; w < words && w < (int)(threadIdx.x + 1) * per; ++w) used_here += __popc(bits[w]);
  int before;
  const int slice = cta_prefix(used_here, s_warp, before);
  if (threadIdx.x < CTAS) G::map(s_totals, threadIdx.x)[rank] = slice;
  G::sync();
  int live = 0;
  for (int i = 0; i < CTAS; ++i) {
    if (i < rank) before += s_totals[i];
    live += s_totals[i];
  }
  for (int w = threadIdx.x * per, x = before; w < words && w < (int)(threadIdx.x + 1) * per; ++w) {
    front[w] = x;
    x += __popc(bits[w]);
  }
  G::sync();
  // Pages in use in front of page number `id`.
  const auto used_before = [&](int id) {
    const int w = id >> 5, at = w & (words - 1), in = w >> a.words_shift;
    if (in >= CTAS) return live;
    return G::map(front, in)[at] + __popc(G::map(bits, in)[at] & ((1u << (id & 31)) - 1));
  };
  const int kept = used_before(live), moves = live - kept;  // in use below `live`; holes there = live - kept
  // A warp writes a word's holes and movers, each lane one of its bits.
  const int lane = lane_id();
  for (int w = threadIdx.x / kWarp; w < words; w += kWarps) {
    const unsigned used = bits[w];
    const int id = (((rank << a.words_shift) + w) << 5) + lane;
    const int here = front[w] + __popc(used & lanemask_lt());  // in use in front of the lane's page
    if (used >> lane & 1) {
      if (id >= live) a.src[here - kept] = id;
    } else if (id < live) {
      a.dst[id - here] = id;
    }
  }
  for (int i = moves + rank * kThreads + (int)threadIdx.x; i < a.num_pages / 2; i += CTAS * kThreads)
    a.src[i] = a.dst[i] = -1;
  if (rank == 0 && threadIdx.x == 0) *a.count = moves;
  G::sync();
  // Entries at or above `live` get their new numbers: each thread those that it wrote itself.
  const int total = a.rows * a.new_width;
  for (int i0 = rank * kThreads + (int)threadIdx.x; i0 < total; i0 += kBatch * CTAS * kThreads) {
    int id[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int i = i0 + e * CTAS * kThreads;
      id[e] = i < total ? a.new_table[i] : -1;
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (id[e] >= live) id[e] = __ldcg(a.dst + (used_before(id[e]) - kept)); else id[e] = -1;
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (id[e] >= 0) a.new_table[i0 + e * CTAS * kThreads] = id[e];
  }
  if (CTAS > 1) G::sync();  // no CTA leaves while others use its shared memory
}

constexpr int kCtas = 8;
// One CTA needs no cluster's barriers, but one SM reads the table alone (with copies, 16 rows of 65: 6.6 us against 9;
// 256 rows of 52: 36 against 30).
bool one_cta(int64_t entries, int64_t num_pages) { return entries <= 4096 && num_pages <= 32768; }

int words_shift_of(int64_t num_pages, int ctas) {
  const int64_t words = (num_pages + 31) / 32;
  int s = 0;
  while (((int64_t)ctas << s) < words) ++s;
  return s;
}

int launch_table(void (*k)(TableArgs), std::atomic<bool>* raised, const TableArgs& a, int ctas, size_t smem, cudaStream_t s) {
  if (!allow_smem(k, raised)) return MOE_ERR_CUDA;
  launch(k, dim3(ctas), dim3(kThreads), smem, s, a);
  return check_launch();
}

bool table_ok(int64_t table_stride, int64_t table_width, int64_t num_seqs, int32_t page_size, int64_t num_pages) {
  return num_seqs >= 0 && table_width >= 0 && page_size >= 1 && num_pages >= 0 && (num_seqs < 2 || table_stride >= table_width);
}
bool table_supported(int64_t table_width, int64_t num_seqs, int32_t page_size, int64_t num_pages) {
  return num_seqs <= MOE_CACHE_MAX_ROWS && num_pages <= MOE_CACHE_MAX_PAGES && table_width <= INT32_MAX &&
         table_width * page_size <= INT32_MAX;
}
int set_table(TableArgs& a, const int32_t* table, int64_t stride, int64_t width, const int32_t* lengths, int64_t seqs, int64_t rows,
              int64_t new_width, int32_t page_size, int64_t num_pages) {
  const int ctas = one_cta(rows * new_width, num_pages) ? 1 : kCtas;
  a.table = table;
  a.table_stride = stride;
  a.width = (int32_t)width;
  a.lengths = lengths;
  a.seqs = (int32_t)seqs;
  a.rows = (int32_t)rows;
  a.new_width = (int32_t)new_width;
  a.page = Divisor((uint32_t)page_size);
  a.columns = Divisor((uint32_t)(new_width < 1 ? 1 : new_width));
  a.num_pages = (int32_t)num_pages;
  a.words_shift = words_shift_of(num_pages, ctas);
  a.whole = ctas > 1 && (ctas << a.words_shift) <= 8192;
  return ctas;
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
// Of a page, for a CTA at a time: four vectors of 32 bytes a thread (0.6 GB moved: 186 us, with 16 bytes and 16 KB 197).
constexpr int64_t kPieceBytes = 32768;

// Four vectors of a thread on their way together.
template <typename V> __device__ __forceinline__ void copy_piece(const char* in, char* out, int64_t bytes) {
  const int n = (int)(bytes / (int64_t)sizeof(V));
  const V* from = reinterpret_cast<const V*>(in);
  V* to = reinterpret_cast<V*>(out);
  for (int k = threadIdx.x; k < n; k += 4 * kCopyThreads) {
    V v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (k + e * kCopyThreads < n) v[e] = ld_stream(from + k + e * kCopyThreads);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (k + e * kCopyThreads < n) to[k + e * kCopyThreads] = v[e];
  }
}

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
    const uintptr_t all = reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out) | (uintptr_t)bytes;
    if ((all & 31) == 0) {
      copy_piece<u32x8>(in, out, bytes);
    } else if ((all & 15) == 0) {
      copy_piece<uint4>(in, out, bytes);
    } else if ((all & 3) == 0) {
      copy_piece<uint32_t>(in, out, bytes);
    } else if ((all & 1) == 0) {
      copy_piece<uint16_t>(in, out, bytes);
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
  a.page = Divisor((uint32_t)cache->page_size);
  // Heads that lie side by side on both sides are one row.
  int64_t row_bytes = (int64_t)cache->head_dim * eb, rows = cache->num_kv_heads;
  if (rows > 1 && a.head_stride == row_bytes && a.k_head == row_bytes && a.v_head == row_bytes) {
    row_bytes *= rows;
    rows = 1;
  }
  if (rows == 1) a.head_stride = a.k_head = a.v_head = 0;
  // Vectors as wide as every row's start and length allow.
  const int64_t all = row_bytes | a.page_stride | a.token_stride | a.head_stride | a.k_row | a.k_head | a.v_row | a.v_head |
                      (int64_t)(reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                                reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const auto go = [&](auto kernel, int vb) {
    a.per_row = Divisor((uint32_t)(row_bytes / vb));
    a.per_token = Divisor((uint32_t)(row_bytes / vb * rows));
    // Up to 256 vectors at a time, eight tokens at most, and 32 warps' work for every SM first (100000 tokens of
    // two heads of 64: 51 us with one token at a time).
    int64_t together = 256 / a.per_token.d, each = num_tokens / ((int64_t)num_sms() * 32);
    together = together < each ? together : each;
    a.together = (int32_t)(together < 1 ? 1 : together > 8 ? 8 : together);
    const int64_t ctas = (num_tokens + 8 * a.together - 1) / (8 * a.together);
    launch(kernel, dim3((unsigned)(ctas < 65535 ? ctas : 65535)), dim3(256), 0, s, a);
  };
  if (all % 16 == 0) go(cache_write_kernel<16>, 16);
  else if (all % 8 == 0) go(cache_write_kernel<8>, 8);
  else if (all % 4 == 0) go(cache_write_kernel<4>, 4);
  else go(cache_write_kernel<2>, 2);
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
      num_rows * new_width > INT32_MAX - kBatch * kCtas * kThreads || grow > INT32_MAX)
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
  const int ctas = set_table(a, page_table, table_stride, table_width, lengths, num_seqs, num_rows, new_width, page_size, num_pages);
  a.parents = parents;
  a.new_table = new_table;
  a.new_lengths = new_lengths;
  a.src = src;
  a.dst = dst;
  a.status = d_status;
  a.grow = grow;
  a.hash_bits = 1;
  while ((1 << a.hash_bits) < 2 * num_rows) ++a.hash_bits;
  const size_t words = (size_t)1 << a.words_shift, hash = (size_t)2 << a.hash_bits;
  a.whole_at = (int32_t)(words + 4 * num_rows + (hash > words ? hash : words));
  const size_t smem = 4 * ((size_t)a.whole_at + (a.whole ? words * kCtas : 0));
  static std::atomic<bool> raised[2][kSmemDevices];
  return launch_table(ctas == 1 ? cache_fork_kernel<1> : cache_fork_kernel<kCtas>, raised[ctas > 1], a, ctas, smem, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_cache_compact(const int32_t* page_table, int64_t table_stride, int64_t table_width,
                                 const int32_t* lengths, int64_t num_seqs, int32_t page_size, int64_t num_pages,
                                 int32_t* new_table, int32_t* src, int32_t* dst, int32_t* count, int32_t* d_status,
                                 moe_stream_t stream) {
  if (!table_ok(table_stride, table_width, num_seqs, page_size, num_pages)) return MOE_ERR_INVALID_ARG;
  if (!table_supported(table_width, num_seqs, page_size, num_pages) || num_seqs * table_width > INT32_MAX - kBatch * kCtas * kThreads)
    return MOE_ERR_UNSUPPORTED;
  if ((num_seqs > 0 && (lengths == nullptr || (table_width > 0 && (page_table == nullptr || new_table == nullptr)))) ||
      (num_pages > 1 && (src == nullptr || dst == nullptr)) || count == nullptr)
    return MOE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)page_table, (const void*)lengths, (const void*)new_table, (const void*)src, (const void*)dst,
                        (const void*)count, (const void*)d_status})
    if (!aligned(p, 4)) return MOE_ERR_UNSUPPORTED;
  TableArgs a = {};
  const int ctas = set_table(a, page_table, table_stride, table_width, lengths, num_seqs, num_seqs, table_width, page_size, num_pages);
  a.new_table = new_table;
  a.src = src;
  a.dst = dst;
  a.count = count;
  a.status = d_status;
  const size_t words = (size_t)1 << a.words_shift;
  a.whole_at = (int32_t)(2 * words + 2 * num_seqs);
  static std::atomic<bool> raised[2][kSmemDevices];
  return launch_table(ctas == 1 ? cache_compact_kernel<1> : cache_compact_kernel<kCtas>, raised[ctas > 1], a, ctas,
                      4 * ((size_t)a.whole_at + (a.whole ? words * kCtas : 0)), reinterpret_cast<cudaStream_t>(stream));
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
    if (caches[c].page_bytes > 65535 * kPieceBytes) return MOE_ERR_UNSUPPORTED;
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
