/* Serving from a paged 8-bit key/value cache (C ABI of the GB300 library).
 *
 * Companion of attn_bwd.h: the same types, status codes and conventions
 * (caller-owned buffers, work queued on ``stream``, every argument checked
 * before anything is queued).  Three operators, used in this order by each
 * step of a server:
 *
 *   attn_kv_block_tables  pages, slots, positions and row ranges of the new
 *                         tokens, from the request lengths, on the device
 *   attn_kv_cache_write   their keys and values into the cache, as e4m3
 *   attn_fwd_kv_cache     attention of their queries over the cached tokens
 *
 * The cache holds ``num_blocks`` pages of ``page_size`` tokens.  A stored byte
 * is an e4m3 value (1 sign, 4 exponent, 3 fraction bits, bias 7, largest 448,
 * no infinities) and stands for byte * scale[page, KV head], K and V with
 * scales of their own.  A request's tokens lie in the pages that its row of
 * the block table lists: position p is token p % page_size of page
 * table[p / page_size].  A slot is page * page_size + token. */
#ifndef ATTN_KV_CACHE_H
#define ATTN_KV_CACHE_H

#include "attn_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The cache.  k, v : e4m3 bytes addressed as base + b*st.b + s*st.s + h*st.h + d
 * (page, token in the page, KV head; the head-dim stride is 1), bases and
 * strides multiples of 16 bytes, so that pages stored token by token
 * [num_blocks, page_size, HKV, D] and head by head [num_blocks, HKV, page_size,
 * D] both serve.  k_scale, v_scale : f32 [num_blocks, HKV], contiguous; scales
 * of pages in use are finite and not negative.  page_size in {16, 32, 64, 128},
 * D in {64, 128}, num_blocks * page_size and num_blocks * HKV below 2^31. */
typedef struct {
  void* k;
  attn_strides_t sk;
  void* v;
  attn_strides_t sv;
  float* k_scale;
  float* v_scale;
  int64_t num_blocks, page_size, HKV, D;
} attn_kv_cache_t;

/* Extends the block table by the pages that new tokens need and gives each new
 * token its slot.  Request n holds ctx_lens[n] tokens and gets new_lens[n]
 * (negative lengths count as 0), with
 *   before_n = ceil(ctx_n / P), after_n = ceil((ctx_n + new_n) / P),
 *   first_n  = sum over m < n of (after_m - before_m):
 *   table[n, before_n + j] = free_blocks[free_start + first_n + j]
 *   cu_seqlens[n + 1]      = cu_seqlens[n] + new_n,  cu_seqlens[0] = 0
 *   kv_lens[n]             = ctx_n + new_n
 *   token t of request n (cu_seqlens[n] <= t < cu_seqlens[n + 1]):
 *     positions[t] = ctx_n + t - cu_seqlens[n]
 *     slot_map[t]  = table[n, positions[t] / P] * P + positions[t] % P
 * Other table entries stay as they are.  slot_map and positions have
 * max_tokens rows; rows past the last token get slot -1 and position 0, so a
 * captured step keeps its shapes.
 *   counts[0] = the new tokens of all requests, counts[1] = pages taken from
 *   the free list, counts[2] = 0 if everything fitted, else the pages that the
 *   free list or the table's width could not give plus the tokens past
 *   max_tokens.  A page that is lacking gets table entry -1 (inside the
 *   table's width) and its tokens slot -1; cu_seqlens stops at max_tokens.  A
 *   plan with counts[2] != 0 is not meant to be run, but the other two
 *   operators stay inside their buffers with it.
 *   ctx_lens, new_lens, kv_lens : int32 [num_seqs];  cu_seqlens : int32
 *   [num_seqs + 1];  block_table : int32 [num_seqs, max_blocks], row stride
 *   table_stride;  free_blocks : int32 [num_free], distinct pages that no table
 *   row holds (an entry outside [0, num_blocks) is taken as -1 and not counted
 *   as lacking);  free_start :
 *   int32 [1] on the device, the first free_blocks entry not yet taken, or NULL
 *   for 0 (a server adds counts[1] to it after the step);  slot_map, positions :
 *   int32 [max_tokens];  counts : int32 [3].  All device memory; the outputs overlap
 *   no input (free_blocks and block_table among them) and not each other.
 * One launch; the result does not depend on the order in which blocks run.
 * Errors: ATTN_ERR_INVALID_ARG (null or misaligned pointer, bad size),
 * ATTN_ERR_UNSUPPORTED (page size, sizes past 2^31), ATTN_ERR_LAUNCH. */
ATTN_BWD_API attn_status_t attn_kv_block_tables(const int32_t* ctx_lens, const int32_t* new_lens, int64_t num_seqs,
                                                int32_t* block_table, int64_t table_stride, int64_t max_blocks,
                                                const int32_t* free_blocks, int64_t num_free,
                                                const int32_t* free_start, int64_t page_size, int64_t num_blocks,
                                                int64_t max_tokens, int32_t* cu_seqlens, int32_t* kv_lens,
                                                int32_t* slot_map, int32_t* positions, int32_t* counts,
                                                void* stream);

/* Writes T new tokens' keys and values into the cache.  Token t goes to slot
 * slot_map[t]; tokens whose slot lies outside [0, num_blocks * page_size) are
 * skipped.  Tokens of one page with ascending slots, no more than 32 tokens
 * apart and with nothing but skipped tokens between them, form a run; a run
 * that starts at token ``off`` of its page appends to the ``off`` tokens that
 * the page holds already (off = 0 starts the page anew).  Per run, head and
 * tensor, with amax the largest finite |x| of the run:
 *   want  = the least power of two s >= 2^-100 with amax <= 448 s
 *   scale = off > 0 ? max(scale, want) : want
 *   where that raises the scale of a page that holds tokens, their bytes are
 *   rounded again, e4m3(byte * old / new);  y = e4m3(x / scale)
 * e4m3() rounds to nearest, ties to even; infinities become +-448, NaN stays.
 * With powers of two, a page's older values keep every bit through a raise
 * unless they drop below the e4m3 normal range of the new scale.  Bytes of the
 * page that the run skips or that lie behind it are left as they were.  One
 * call's runs go to different pages (as slots of attn_kv_block_tables do):
 * where two runs of a call share a page, that page's contents are unspecified,
 * and nothing else is touched.
 *   k, v : [1,T,HKV,D] 16-bit (strides b unused);  slot_map : int32 [T].
 * T = 0 queues nothing.  Errors: ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED
 * (dtype, head dim, page size, T above 2^31 - 4096), ATTN_ERR_LAUNCH. */
ATTN_BWD_API attn_status_t attn_kv_cache_write(const void* k, attn_strides_t sk, const void* v, attn_strides_t sv,
                                               const int32_t* slot_map, int64_t T, attn_dtype_t dtype,
                                               const attn_kv_cache_t* cache, void* stream);

/* Bytes of workspace attn_fwd_kv_cache needs for T queries: the 256-byte
 * header and the f32 partials of rows whose keys are split over CTAs (0 for
 * sizes that it refuses). */
ATTN_BWD_API size_t attn_fwd_kv_cache_workspace_size(int64_t T, int64_t HQ, int64_t HKV, int64_t D);

/* O = softmax(sm_scale Q K^T) V and the natural-log LSE over cached keys.
 * Packed queries: request n owns rows [cu_seqlens[n], cu_seqlens[n + 1]) of q
 * (clamped to [0, T]), nq_n of them, and sees the first kv_lens[n] positions of
 * its block-table row (its new tokens are in the cache already).  Query i of
 * the request stands at position i + kv_lens[n] - nq_n, as attn_mask_t aligns
 * rows of unequal length, and sees key j < kv_lens[n] iff
 *   causal == 0 and window_left < 0 : always (cross attention to cached states)
 *   causal != 0                     : j <= its position
 *   window_left = W > 0             : its position - W < j <= its position
 * Keys past the table's width (max_blocks * page_size) or in a page whose
 * table entry lies outside [0, num_blocks) are not visible.  A query that sees
 * no key gets O = 0 and LSE = -inf.  Cached bytes and scales that no query of
 * the request sees are never used as operands: they may hold anything, NaN
 * included.  (A NaN that one query of a request sees may make others of it NaN,
 * as 0 * NaN does.)  Rows of q past cu_seqlens[num_seqs] are not written.
 * q, o : [1,T,HQ,D] 16-bit (strides b unused);  lse : f32, lse[h*slse.h +
 * t*slse.s];  block_table : int32 [num_seqs, max_blocks], row stride
 * table_stride;  cu_seqlens [num_seqs + 1], kv_lens [num_seqs] : int32, device
 * memory;  HQ a multiple of HKV, query head h reads KV head h / (HQ / HKV);
 * sm_scale finite and > 0.
 * The products run on fp16 operands with f32 sums, for either dtype of q: e4m3
 * values are exact in fp16, each q row is brought into fp16's range by a power
 * of two of its own, K scales multiply the f32 scores, and V scales multiply P in
 * f32.  These weights, P vs, are rounded to fp16 once, after a power of two of the
 * row's own that follows its largest one: V scales of any spread serve, up to 2^70
 * (rows of split keys are summed before they are divided by l), and what a row
 * does not see, or gives no weight, costs it nothing.  (Rows whose weights are all
 * below 2^-100 lose bits.)  Weights below 2^-21 (few rows: queries
 * * heads of a group) or 2^-17 (many) of the row's largest are held in steps of 2^-31
 * or 2^-27 of it.
 * One kernel is made for requests of few rows and another for many; either serves
 * any.  No length is needed on the host: it queues one of them or both by the mean
 * of rows a request, T (padding rows included) * HQ / HKV / num_seqs, so that a request
 * far from its batch's mean may run in the slower one (both from 16 to 259; below, a
 * long chunk beside many single tokens takes up to five times its time).  Rows whose keys
 * were split over CTAs are joined by a last launch.  Pages may
 * be listed by several requests, and twice by one.  o, lse and the workspace
 * overlap no input and not each other.
 *   workspace : attn_fwd_kv_cache_workspace_size(T, HQ, HKV, D) bytes, 16-byte
 *   aligned, owned by the caller until the work is done; its contents on entry
 *   do not matter; attn_bwd_check_error reports a kernel whose bounded wait ran
 *   out.
 * T = 0 queues nothing.  Errors: ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED
 * (dtype, head dim, page size, T * HQ or max_blocks * page_size above
 * 2^31 - 4096, more than 2^20 requests), ATTN_ERR_WORKSPACE before anything is
 * queued; ATTN_ERR_LAUNCH. */
ATTN_BWD_API attn_status_t attn_fwd_kv_cache(const void* q, attn_strides_t sq, int64_t T, int64_t HQ,
                                             attn_dtype_t dtype, float sm_scale, const attn_kv_cache_t* cache,
                                             const int32_t* block_table, int64_t table_stride, int64_t max_blocks,
                                             const int32_t* cu_seqlens, const int32_t* kv_lens, int64_t num_seqs,
                                             int32_t causal, int32_t window_left, void* o, attn_strides_t so,
                                             float* lse, attn_strides_t slse, void* workspace,
                                             size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_KV_CACHE_H */
