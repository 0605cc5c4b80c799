/* Rotary positions of queries and keys (C ABI of the GB300 library).
 *
 * Companion of attn_bwd.h: the same types, status codes and conventions.  The
 * operator stands before attention (the forwards of attn_bwd.h, the cache
 * write of attn_kv_cache.h) and, inverted, behind its backward. */
#ifndef ATTN_ROPE_H
#define ATTN_ROPE_H

#include "attn_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One tensor to rotate: x and y are [B,S,H,D] 16-bit, addressed as base + b*st.b
 * + s*st.s + h*st.h + d; columns [start, start + rotary_dim) of each head are
 * rotated, the others copied.  y == x with equal strides works in place and
 * leaves the other columns untouched; otherwise x and y do not overlap.  Bases
 * and strides multiples of 16 bytes; D and start multiples of 8, start +
 * rotary_dim <= D. */
typedef struct {
  const void* x;
  attn_strides_t sx;
  void* y;
  attn_strides_t sy;
  int64_t H, D, start;
} attn_rope_tensor_t;

/* Turns pair i of every head at position p by the angle t = 2 pi p steps[i] /
 * 2^64 and scales it:
 *   y1 = scale (x1 cos t - x2 sin t),  y2 = scale (x1 sin t + x2 cos t)
 * with (x1, x2) the columns start + i and start + i + rotary_dim / 2 (the half
 * layout) or start + 2i and start + 2i + 1 (interleaved != 0); inverse != 0 turns by -t,
 * the gradient of x given that of y.  The frequencies are fractions of a turn a
 * position as 64-bit fixed point: p * steps[i] keeps its fraction of a turn
 * exactly, so that far positions lose nothing (an f32 angle at 10^6 is off by
 * 2^-5 radians); the angle itself is f32, within 2^-26 turns.  The products and sums are
 * f32, rounded once.
 *   q : a tensor;  k : another one with heads and columns of its own, or NULL (both
 *   take one launch)
 *   positions : int32, of row b at positions + b * positions_b (0: all rows
 *   alike), S each; any value, negative ones turn backwards
 *   steps : uint64 [rotary_dim / 2], device memory;  scale finite
 *   rotary_dim : a multiple of 16, at most 1024
 * S = 0 queues nothing.  Errors: ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED
 * (dtype, rotary_dim, D above 1024, B * S or B * S * H past 2^31, more than 2^20 heads), ATTN_ERR_LAUNCH. */
ATTN_BWD_API attn_status_t attn_rope(const attn_rope_tensor_t* q, const attn_rope_tensor_t* k, int64_t B, int64_t S,
                                     attn_dtype_t dtype, const int32_t* positions, int64_t positions_b,
                                     const uint64_t* steps, int64_t rotary_dim, float scale, int32_t interleaved,
                                     int32_t inverse, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_ROPE_H */
