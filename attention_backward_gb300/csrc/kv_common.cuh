// Device helpers of attention over the 8-bit cache.
#pragma once
#include "cvt.cuh"
#include "kv_cache.h"

namespace ab {

// Four e4m3 bytes -> two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t* lo, uint32_t* hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(*lo), "=r"(*hi)
      : "r"(w));
}

// Power of two that brings a largest absolute value into [2^14, 2^15), and its
// inverse; 1 for 0, infinities and NaN.
__device__ __forceinline__ float to_top(float amax, float* back) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23);  // biased
  if (!(amax > 0.f) || e == 255) {
    *back = 1.f;
    return 1.f;
  }
  int up = 14 - (e - 127);
  up = up > 126 ? 126 : up;  // subnormal rows
  *back = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
}

// The weight of key j in O_i is p_ij vs_j, p = 2^(x - m_i) and vs its page's V scale.
// It is rounded to fp16 as p vs 2^ref_i, ref_i a whole number of the row's own: where
// it is set, the row's largest weight so far lands in (2^(top - 1), 2^top], top being the
// kernel's.  Below fp16's normal range, from 2^(-14 - top) of that largest on, a weight
// keeps the steps of 2^(-24 - top) of it; above, there is room to grow before ref is
// set anew.  (Set for a whole unit by its pages' largest V scale, ref let the weights of
// rows that do not see that page, or give it none, fall below fp16's range.  At a top
// of 0, the many small weights beside one large one, a sink, were lost from 2^-25 on,
// while l counted them whole.)
constexpr float kKvRefNone = 100.f;  // of a row that has met no weight above 2^-100, the smallest scale of a write
__device__ __forceinline__ float weight_ref(float top, float log2_top) {
  return fminf(fmaxf(top - ceilf(log2_top), -126.f), kKvRefNone);
}
// 2^(log2 vs + ref), finite also where a row without weights meets a large scale
// (its p are then tiny or 0).
__device__ __forceinline__ float weight_factor(float log2_vs, float ref) { return ex2(fminf(log2_vs + ref, 126.f)); }

// Writes of one row's final O (16-bit, ND values from column d0) and LSE.
template <bool BF16, int ND>
__device__ __forceinline__ void store_o(const KvAttnParams& p, int64_t t, int hq, int d0, const float* o) {
  uint8_t* out = p.o + 2 * (t * p.so_s + static_cast<int64_t>(hq) * p.so_h + d0);
  if constexpr (ND >= 8) {
#pragma unroll
    for (int i = 0; i < ND; i += 8) {
      uint4 w;
      w.x = pack2<BF16>(o[i], o[i + 1]), w.y = pack2<BF16>(o[i + 2], o[i + 3]);
      w.z = pack2<BF16>(o[i + 4], o[i + 5]), w.w = pack2<BF16>(o[i + 6], o[i + 7]);
      *reinterpret_cast<uint4*>(out + 2 * i) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < ND; i += 2) *reinterpret_cast<uint32_t*>(out + 2 * i) = pack2<BF16>(o[i], o[i + 1]);
  }
}

// m in log2 units; a row that saw no key has l = 0.
__device__ __forceinline__ void store_lse(const KvAttnParams& p, int64_t t, int hq, float m, float l) {
  p.lse[hq * p.sl_h + t * p.sl_s] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Byte offset of 16-byte chunk ``c`` of row ``r`` in a tile of D-byte rows, as
// the copies' 128-byte (D = 128) or 64-byte (D = 64) swizzle places it.
template <int D>
__device__ __forceinline__ int kv_chunk_at(int r, int c) {
  return r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

}  // namespace ab
