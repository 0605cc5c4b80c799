/* Latent attention (C ABI of the GB300 library): keys and values from one row
 * a token that all heads share.
 *
 * Companion of attn_bwd.h: the same types, status codes and conventions.  A
 * latent row has 576 16-bit values: the latent vector c (512), which stands for
 * keys and values, and a rotated key part k of 64 columns (attn_rope.h).
 *
 *   attn_latent_cache_write  rows of new tokens into a paged cache, c normalised
 *                            and k rotated on the way
 *   attn_fwd_latent_cache    attention over the cache in the absorbed form: the
 *                            heads' key and value projections are in q and behind o
 *   attn_fwd_sparse          the same over index lists: O and LSE of top-k sparse
 *                            attention, as attn_bwd_sparse takes them
 *   attn_fwd_latent          the expanded form for prompts: keys of 128 columns and
 *                            values of 128 a head, beside the shared k
 *
 * Pages and slots are those of attn_kv_block_tables (attn_kv_cache.h). */
#ifndef ATTN_LATENT_H
#define ATTN_LATENT_H

#include "attn_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_LATENT_ROW 576 /* values of a row */
#define ATTN_LATENT_DIM 512 /* of them the latent vector */

/* The cache: slot s (page s / page_size, token s % page_size) holds the 16-bit
 * row at rows + s * row_stride (elements).  Base and row_stride multiples of 16
 * bytes, row_stride >= 576, page_size in {16, 32, 64, 128}, num_blocks *
 * page_size below 2^31. */
typedef struct {
  void* rows;
  int64_t row_stride;
  int64_t num_blocks, page_size;
} attn_latent_cache_t;

/* Writes T rows (c | k) into the cache:
 *   c' = c / sqrt(mean(c^2) + norm_eps) * norm_weight   (norm_weight NULL: c)
 *   k' = k turned to its token's position as by attn_rope  (steps NULL: k)
 *   row slot_map[t] = (c' | k')
 * Sums and products in f32, each value rounded once.  Tokens whose slot lies
 * outside [0, num_blocks * page_size) leave the cache alone; where two tokens of
 * a call share a slot, its row is one value of either, column by column.
 *   kv : row t at kv + t * kv_stride (elements; 16-byte multiples, >= 576)
 *   slot_map : int32 [T];  norm_weight : 16-bit [512];  norm_eps >= 0
 *   positions : int32 [T], steps : uint64 [32] (both or neither)
 *   rope_scale, interleaved : as attn_rope's
 *   out : NULL, or rows that get (c' | k') of every token too, skipped ones
 *   among them (a prompt's own expanded keys and values are made from them); kv
 *   itself with out_stride = kv_stride serves; otherwise it overlaps nothing.
 * T = 0 queues nothing.  Errors: ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED
 * (dtype, page size, T above 2^31 - 4096), ATTN_ERR_LAUNCH. */
ATTN_BWD_API attn_status_t attn_latent_cache_write(const void* kv, int64_t kv_stride, const int32_t* slot_map,
                                                   int64_t T, attn_dtype_t dtype, const void* norm_weight,
                                                   float norm_eps, const int32_t* positions, const uint64_t* steps,
                                                   float rope_scale, int32_t interleaved,
                                                   const attn_latent_cache_t* cache, void* out, int64_t out_stride,
                                                   void* stream);

/* Bytes of workspace attn_fwd_latent_cache needs: a 256-byte header and the
 * f32 partials of rows whose keys are split over CTAs. */
ATTN_BWD_API size_t attn_fwd_latent_cache_workspace_size(void);

/* O = softmax(sm_scale q (c | k)^T) c and the natural-log LSE over cached rows.
 * Packed queries and block tables as attn_fwd_kv_cache has them: request n owns
 * rows [cu_seqlens[n], cu_seqlens[n + 1]) of q (clamped to [0, T]), nq_n of them, and
 * sees the first kv_lens[n] positions of its table row; query i stands at position
 * i + kv_lens[n] - nq_n and sees key j < kv_lens[n] iff causal == 0 or j <= its
 * position.  Keys past the table's width or in a page whose entry lies outside [0,
 * num_blocks) are not visible.  A query that sees no key gets O = 0 and LSE = -inf.
 * Cached rows that no query of the request sees are never used as operands.  (A NaN
 * that one query of a request sees may make others of it NaN, as 0 * NaN does.)  Rows of
 * q past cu_seqlens[num_seqs] are not written.
 *   q : [1,T,H,576], o : [1,T,H,512] 16-bit of the cache's type (strides b unused)
 *   lse : f32, lse[h*slse.h + t*slse.s];  block_table : int32 [num_seqs,
 *   max_blocks], row stride table_stride;  cu_seqlens [num_seqs + 1], kv_lens
 *   [num_seqs] : int32, device memory;  sm_scale finite and > 0
 * Scores and sums are f32; a weight is rounded to the 16-bit type once, and l sums
 * the f32 weights.  No length is needed on the host.  Rows whose keys were split
 * over CTAs are joined by a second launch in a fixed order.  o, lse and the workspace
 * overlap no input and not each other.
 *   workspace : attn_fwd_latent_cache_workspace_size() bytes, 16-byte aligned,
 *   owned by the caller until the work is done; attn_bwd_check_error reports a
 *   kernel whose bounded wait ran out.
 * T = 0 queues nothing.  Errors: ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED
 * (dtype, page size, T * H or max_blocks * page_size above 2^31 - 4096, more than
 * 2^20 requests), ATTN_ERR_WORKSPACE before anything is queued; ATTN_ERR_LAUNCH. */
ATTN_BWD_API attn_status_t attn_fwd_latent_cache(const void* q, attn_strides_t sq, int64_t T, int64_t H,
                                                 attn_dtype_t dtype, float sm_scale, const attn_latent_cache_t* cache,
                                                 const int32_t* block_table, int64_t table_stride, int64_t max_blocks,
                                                 const int32_t* cu_seqlens, const int32_t* kv_lens, int64_t num_seqs,
                                                 int32_t causal, void* o, attn_strides_t so, float* lse,
                                                 attn_strides_t slse, void* workspace, size_t workspace_bytes,
                                                 void* stream);

/* Bytes of workspace with which attn_fwd_sparse may split the lists of few tokens
 * over CTAs: the 256-byte header and their f32 partials (256 where it would not). */
ATTN_BWD_API size_t attn_fwd_sparse_workspace_size(int64_t B, int64_t S, int64_t HKV);

/* The forward of attn_bwd_sparse: per query head h of KV group g = h / (H / HKV)
 * and token t, over the rows that the list idx[b, t, g, :] names,
 *   O = softmax(sm_scale q kv_row^T) kv_row[:DV] and the natural-log LSE.
 * Entries outside [0, SKV) are not visible and never dereferenced, repeated ones
 * count once a slot; a list without a visible entry gives O = 0 and LSE = -inf.
 * Scores and sums are f32; a weight is rounded to the 16-bit type once, and l sums the
 * f32 weights.
 *   q : [B,S,H,576], kv : [B,SKV,HKV,576], o : [B,S,H,512] 16-bit;  the rows of kv are
 *   evenly spaced (skv.s = HKV skv.h, skv.b = SKV skv.s);  idx : int32
 *   [B,S,HKV,topk], strides sidx, unit slot stride;  lse : f32, lse[b*slse.b +
 *   h*slse.h + s*slse.s];  H / HKV at most 64;  DQK = 576, DV = 512;  sm_scale finite and
 *   > 0.
 *   workspace : at least 256 bytes, 16-byte aligned (a backward workspace serves; with
 *   attn_fwd_sparse_workspace_size bytes the lists of few tokens are split, and joined by
 *   a second launch in a fixed order).
 * Errors as attn_bwd_sparse's. */
ATTN_BWD_API attn_status_t attn_fwd_sparse(const void* q, attn_strides_t sq, const void* kv, attn_strides_t skv,
                                           const int32_t* idx, attn_strides_t sidx, int64_t B, int64_t S, int64_t SKV,
                                           int64_t H, int64_t HKV, int64_t DQK, int64_t DV, int64_t topk,
                                           attn_dtype_t dtype, float sm_scale, void* o, attn_strides_t so, float* lse,
                                           attn_strides_t slse, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace attn_fwd_latent needs for S queries a batch row (num_seqs: packed
 * sequences, 0 for dense rows): the 256-byte header, and, where the queries are few,
 * the f32 partials of rows whose keys are split over CTAs.  0 for sizes that it refuses. */
ATTN_BWD_API size_t attn_fwd_latent_workspace_size(int64_t B, int64_t S, int64_t H, int64_t num_seqs);

/* The expanded form: head h has keys (kn_h | kr), 128 columns of its own and 64
 * that all heads share, and values v_h of 128:
 *   O = softmax(sm_scale (qn kn_h^T + qr kr^T)) v_h and the natural-log LSE
 * under the mask of attn_fwd_gqa (causal, packed sequences, kv_len; no window:
 * window_left must be -1).
 *   q : [B,S,H,192] (qn | qr), kn, v : [B,Sk,H,128] (columns of one projection: any
 *   strides of 16-byte multiples), kr : [B,Sk,64] (strides skr.b, skr.s), o :
 *   [B,S,H,128] 16-bit;  lse : f32, lse[b*slse.b + h*slse.h + s*slse.s]
 * Scores and sums are f32; a weight is rounded to the 16-bit type once, and l sums the
 * f32 weights.  A query that sees no key gets O = 0 and LSE = -inf.  Rows past
 * cu_seqlens[num_seqs] are not written and may hold anything.  (A NaN in a row of v that
 * some query of a sequence sees may make others of it NaN, as 0 * NaN does.)
 *   workspace : attn_fwd_latent_workspace_size(B, S, H, num_seqs) bytes, 16-byte
 *   aligned.  Rows whose keys were split are joined by a second launch in a fixed order.
 * Errors as attn_fwd_gqa's. */
ATTN_BWD_API attn_status_t attn_fwd_latent(const void* q, attn_strides_t sq, const void* kn, attn_strides_t skn,
                                           const void* kr, attn_strides_t skr, const void* v, attn_strides_t sv,
                                           int64_t B, int64_t S, int64_t H, attn_dtype_t dtype, float sm_scale,
                                           const attn_mask_t* mask, void* o, attn_strides_t so, float* lse,
                                           attn_strides_t slse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_LATENT_H */
