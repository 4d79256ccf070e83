/*
 * moe_decode.h - C ABI of what a decode step of an MoE model needs around the
 * few-token layer (same library, libmoe_route.so, as moe_route.h and
 * moe_block.h): a key-value cache in pages, the attention of one new token over
 * it, the moves of its pages, and beam search's selection.
 *   moe_cache_fork, moe_cache_copy -> per layer: moe_attention_decode,
 *   moe_layer -> moe_beam_select -> the next step
 *
 * The conventions of moe_route.h hold: device pointers owned by the caller
 * (the structs below and arrays marked so are read on the host, during the call),
 * no allocation, work enqueued on `stream` without a host synchronisation,
 * MOE_* return codes before anything is enqueued, MOE_STATUS_* bits OR-ed into
 * a nullable `d_status`. The current device is the one of the pointers and the
 * stream. Nothing here waits for another kernel's CTAs: every call can be
 * captured into a graph. Calls that may run at the same time need workspaces of
 * their own.
 *
 * The cache. A pool of num_pages pages holds page_size tokens each; row b of a
 * page table (int32, table_width entries, rows table_stride entries apart)
 * names the pages of sequence b in order: its position p is token
 * p % page_size of page table[b][p / page_size]. lengths[b] (int32) is the
 * number of its tokens. Only entries in front of ceil(lengths[b] / page_size)
 * are read, what stands behind them does not matter. Rows may share pages that
 * are full. A page number outside [0, num_pages) where one is needed sets
 * MOE_STATUS_BAD_INDEX and its positions count as absent; a length outside
 * [0, table_width * page_size] sets it and is cut to that range.
 */
#ifndef MOE_DECODE_H
#define MOE_DECODE_H

#include "moe_route.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Another bit of *d_status: the pool had too few free pages, or the table too few columns. */
#define MOE_STATUS_NO_PAGES 32

#define MOE_ATTENTION_MAX_DIM 256
#define MOE_CACHE_MAX_ROWS 4096
#define MOE_CACHE_MAX_PAGES (1 << 22)
#define MOE_CACHE_MAX_CACHES 256
#define MOE_BEAM_MAX_BEAMS 64
#define MOE_BEAM_MAX_OUT 128
#define MOE_BEAM_MAX_UNITS (1 << 15)

/*
 * Keys and values of one layer: token t, head h of page i starts at element
 * i*page_stride + t*token_stride + h*head_stride of k and of v, and its
 * head_dim elements are contiguous. Any strides: tokens first or heads first,
 * slices of a larger tensor.
 */
typedef struct moe_kv_cache {
  void* k;
  void* v;
  int64_t num_pages, page_stride, token_stride, head_stride; /* strides in elements */
  int32_t dtype;                                             /* MOE_F32 or MOE_BF16 */
  int32_t page_size, num_kv_heads, head_dim;
} moe_kv_cache;

/* [rows, heads, head_dim] of the cache's dtype, contiguous in the last dimension (strides in elements). */
typedef struct moe_heads {
  const void* data;
  int64_t row_stride, head_stride;
} moe_heads;

/*
 * Attention of one new token of every sequence over its cache:
 *   s_j = scale * q . k_j, p = softmax(s), out = sum_j p_j v_j,
 *   lse = log sum_j exp(s_j)
 * over the positions j in [max(0, L - window), L) of the sequence, L =
 * lengths[b] with the new token counted; window 0: all of them. A sequence
 * without positions (L = 0) gets +0.0 and lse = -infinity.
 *   q      [num_seqs, num_heads, head_dim]; num_heads is a multiple of
 *          num_kv_heads, and head h reads kv head h / (num_heads / num_kv_heads)
 *   k_new, v_new  [num_seqs, num_kv_heads, head_dim], both or neither: written
 *          to position L - 1 of the cache, and read from here. The page that
 *          takes it belongs to one sequence alone. A token without a place is
 *          left out: its page's number is bad, or its length lies beyond the
 *          table (then only what the table holds is looked at).
 *   out    [num_seqs, num_heads, head_dim] of the cache's dtype, contiguous
 *   lse    [num_seqs, num_heads] fp32, nullable
 *   workspace >= moe_attention_decode_workspace_size(...) bytes, 16-byte aligned, contents need no initialisation;
 *          the size is that of the current device (0 for sizes that the call refuses).
 * Sums and the softmax's statistics are fp32, out is rounded once. bf16 caches
 * run on the tensor cores with the probabilities as sums of two bf16 numbers
 * (16 significant bits). The sums of values are divided last: values whose sum
 * over the positions passes fp32's largest number come out infinite or NaN,
 * although their mean does not. A NaN or +infinity among a head's scores makes
 * its out and lse NaN; a score of -infinity has weight 0, and a head all of
 * whose scores are -infinity counts as one without positions. An infinite value
 * makes its element of out infinite or NaN. A sequence's result depends on the other sequences'
 * lengths in the order of its sums alone; repeated calls give the same bits.
 * head_dim <= MOE_ATTENTION_MAX_DIM, num_seqs <= MOE_CACHE_MAX_ROWS, num_heads
 * <= 2^30, num_pages < 2^31, table_width * page_size < 2^31 - 16 and
 * num_seqs * table_width * page_size < 2^34, else MOE_ERR_UNSUPPORTED.
 */
size_t moe_attention_decode_workspace_size(int64_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                           int32_t head_dim);
int moe_attention_decode(const moe_kv_cache* cache, const moe_heads* q, int32_t num_heads, const int32_t* page_table,
                         int64_t table_stride, int64_t table_width, const int32_t* lengths, int64_t num_seqs,
                         const moe_heads* k_new, const moe_heads* v_new, float scale, int64_t window, void* out,
                         float* lse, void* workspace, size_t workspace_bytes, int32_t* d_status,
                         moe_stream_t stream);

/*
 * Writes keys and values of many tokens (prompts, or pieces of them) into the
 * cache: rows offsets[b] .. offsets[b+1] - 1 of k and v are the last tokens of
 * sequence b, the last one at position lengths[b] - 1.
 *   k, v [num_tokens, num_kv_heads, head_dim]
 *   offsets [num_seqs + 1] int32, ascending from 0; rows from offsets[num_seqs]
 *           on are not read. Offsets that do not ascend or lie outside
 *           [0, num_tokens] set MOE_STATUS_BAD_BINS, and no row outside
 *           [0, num_tokens) is read.
 * A token whose position is negative or lies beyond the table, or whose page is
 * bad, is left out (MOE_STATUS_BAD_INDEX). Nothing else of the cache changes.
 * head_dim <= 2^20, num_kv_heads * head_dim <= 2^26, num_tokens and num_pages
 * < 2^31 and num_seqs < 2^31 - 1, else MOE_ERR_UNSUPPORTED.
 */
int moe_cache_write(const moe_kv_cache* cache, const moe_heads* k, const moe_heads* v, int64_t num_tokens,
                    const int32_t* offsets, const int32_t* page_table, int64_t table_stride, int64_t table_width,
                    const int32_t* lengths, int64_t num_seqs, int32_t* d_status, moe_stream_t stream);

/*
 * The page table of the next step: row r goes on from row parents[r] of the old
 * table, with room for `grow` more tokens (-1: from nothing; an empty row
 * without a page, whatever `grow` is).
 *   new_lengths[r] = lengths[parents[r]] (the tokens to come are not counted)
 *   new_table[r]   = the parent's pages, then fresh ones up to
 *                    ceil((length + grow) / page_size), then -1
 * Rows with the same parent share its pages, but a last page that is not full
 * cannot be written by several: the first row (in order of r) that holds it
 * keeps it, every other one gets a fresh page in its place and the copy
 * src[r] -> dst[r] (-1, -1 where there is none), for moe_cache_copy. With
 * grow = 0 nothing is written, and nothing copied.
 * A page is free when no row of the new table names it: dropping a row frees its
 * pages, and there is no other bookkeeping. Fresh pages go to the requests in
 * order of rows (a row's copied page before its further ones), the i-th request
 * taking the i-th lowest free page. Without enough free pages or columns the
 * remaining requests get -1 (no copy then) and MOE_STATUS_NO_PAGES is set.
 *   page_table, lengths [num_seqs] as above; parents [num_rows] int32: an entry
 *   outside [-1, num_seqs) sets MOE_STATUS_BAD_INDEX and counts as -1
 *   new_table [num_rows, new_width] int32, contiguous; new_lengths, src, dst [num_rows] int32
 * new_width >= table_width. num_seqs and num_rows <= MOE_CACHE_MAX_ROWS, num_pages
 * <= MOE_CACHE_MAX_PAGES, grow and table_width * page_size < 2^31 and
 * num_rows * new_width < 2^31 - 2^15, else MOE_ERR_UNSUPPORTED.
 */
int moe_cache_fork(const int32_t* page_table, int64_t table_stride, int64_t table_width, const int32_t* lengths,
                   int64_t num_seqs, const int32_t* parents, int64_t num_rows, int32_t page_size, int64_t num_pages,
                   int64_t grow, int32_t* new_table, int64_t new_width, int32_t* new_lengths, int32_t* src,
                   int32_t* dst, int32_t* d_status, moe_stream_t stream);

/*
 * Moves the pages in use to the front of the pool: with n of them, the i-th
 * page in use at or above n goes to the i-th unused one below n.
 *   new_table [num_seqs, table_width] int32, contiguous: the table with the new
 *             numbers, -1 behind each row's pages
 *   src, dst  [num_pages / 2] int32: the copies for moe_cache_copy, then -1
 *   count     [1] int32: their number
 * Limits as for moe_cache_fork, with num_seqs rows of table_width.
 */
int moe_cache_compact(const int32_t* page_table, int64_t table_stride, int64_t table_width, const int32_t* lengths,
                      int64_t num_seqs, int32_t page_size, int64_t num_pages, int32_t* new_table, int32_t* src,
                      int32_t* dst, int32_t* count, int32_t* d_status, moe_stream_t stream);

/* One tensor of pages: page i is the page_bytes bytes from i * page_stride on (both in bytes). */
typedef struct moe_cache_pages {
  void* data;
  int64_t page_stride, page_bytes;
} moe_cache_pages;

/*
 * Copies page src[i] to page dst[i] in each of num_caches tensors (a host
 * array; keys and values, every layer), for i < num_copies, or i < *count
 * where count (device, nullable) is smaller. Pairs with a negative number are
 * passed over; numbers from num_pages on too, with MOE_STATUS_BAD_INDEX. All
 * copies read what was there before the call: no page is both a src and a dst,
 * or dst twice.
 * num_caches <= MOE_CACHE_MAX_CACHES, num_pages < 2^31, and less than 2 GB in one
 * page of all of them together (65535 pieces of up to 32 KB, of which a tensor
 * has whole ones), else MOE_ERR_UNSUPPORTED.
 */
int moe_cache_copy(const moe_cache_pages* caches, int64_t num_caches, int64_t num_pages, const int32_t* src,
                   const int32_t* dst, int64_t num_copies, const int32_t* count, int32_t* d_status,
                   moe_stream_t stream);

/*
 * Beam search's selection: with row r = b*num_beams + w for beam w of request b,
 *   total(w, t) = scores[r] + logits[r][t] - log sum_u exp(logits[r][u])
 * the num_out largest totals of each request, largest first, equal ones in
 * order of w*vocab + t.
 *   logits [num_requests * num_beams, vocab] dtype, rows row_stride elements apart
 *   scores [num_requests * num_beams] fp32
 *   ended  [num_requests * num_beams] uint8, nullable: a beam with a nonzero
 *          entry has one candidate, end_token at total = scores[r]; its logits
 *          are not looked at
 *   out_scores fp32, out_parents int32 (row r, such as moe_cache_fork's
 *          parents), out_tokens int32, each [num_requests, num_out]
 *   workspace >= moe_beam_select_workspace_size(...) bytes, 16-byte aligned, contents need no initialisation (0 for sizes
 *          that the call refuses)
 * A logit of -infinity is no candidate, and neither is anything of a beam whose
 * score or log sum is not finite (logits with a NaN or +infinity, or all
 * -infinity). Where candidates run out, score -infinity, parent -1 and token -1.
 * Totals are compared in 48 bits. The log sums come from 32-bit exponentials and
 * sums: off by 5e-8 as a rule (root mean square over vocabularies of 2 to 129280),
 * 4e-7 at most in all that was measured. Totals of one beam come in their order;
 * those of different beams that are nearer than twice that error in either.
 * Repeated calls give the same bits.
 * num_beams <= MOE_BEAM_MAX_BEAMS, num_out <= MOE_BEAM_MAX_OUT, num_beams * ceil(vocab / 512) <= MOE_BEAM_MAX_UNITS
 * and num_requests * num_beams < 2^31, else MOE_ERR_UNSUPPORTED.
 */
size_t moe_beam_select_workspace_size(int64_t num_requests, int32_t num_beams, int64_t vocab);
int moe_beam_select(const void* logits, int32_t dtype, int64_t row_stride, const float* scores, const uint8_t* ended,
                    int64_t num_requests, int32_t num_beams, int64_t vocab, int32_t num_out, int32_t end_token,
                    float* out_scores, int32_t* out_parents, int32_t* out_tokens, void* workspace,
                    size_t workspace_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DECODE_H */
