// How attention over the cache is cut into work: units and their key tiles,
// shared by the kernels and their host checks.
//
// A unit is a row tile (RT consecutive rows of a request, row = query * G +
// head of the group) of one KV head, with the key tiles of KT keys that some
// row of it sees; a unit that sees nothing has one empty tile, so that its
// rows are written.  A head's units, ordered by request and row tile, are laid
// on one line, each as COST positions for its start and end (its table
// row, its queries, its first copies: about as long as that many tiles) and one
// position a tile.  (The prompt kernel has one line for all heads, a row tile's
// heads one after another.)  Part g of C takes the positions [W g / C, W (g + 1) / C) of
// the W: every part gets the same work whatever the lengths, a long row spreads
// over many parts, many short ones share a part, and no length is needed on
// the host.
#pragma once
#include "kv_cache.h"

namespace ab {

struct KvReq {
  int a, nq, L, off, R;  // first row of q, queries, visible key positions, key position of query 0, rows (nq * G)
};

__host__ __device__ __forceinline__ KvReq kv_request(int n, const KvAttnParams& p) {
  KvReq r;
  const int a = clamp_pos(p.cu[n], p.T), e = clamp_pos(p.cu[n + 1], p.T);
  r.a = a;
  r.nq = e > a ? e - a : 0;
  const int len = imax(p.kv_lens[n], 0);
  const int64_t width = static_cast<int64_t>(p.max_blocks) << p.page_log2;
  r.L = len < width ? len : static_cast<int>(width);
  r.off = len - r.nq;
  r.R = r.nq * p.G;
  if (r.R < p.rows_min || r.R > p.rows_max) r.R = 0;  // another kernel's
  return r;
}

// Keys [lo, hi) that query i of a request sees (empty: lo >= hi).
__host__ __device__ __forceinline__ void kv_row_keys(const KvReq& r, int i, int causal, int window, int* lo, int* hi) {
  const int64_t pos = static_cast<int64_t>(r.off) + i;
  int64_t l = 0, h = r.L;
  if (causal || window > 0) h = h < pos + 1 ? h : pos + 1;
  if (window > 0) l = pos - window + 1 > 0 ? pos - window + 1 : 0;
  *lo = static_cast<int>(l < r.L ? l : r.L);
  *hi = static_cast<int>(h < 0 ? 0 : h);
}

struct KvTiles {
  int t0, n;   // first key tile and tiles (at least 1)
  int lo, hi;  // keys that some row of the unit sees
};

// Key tiles of row tile rt of a request.
template <int RT, int KT>
__host__ __device__ __forceinline__ KvTiles kv_row_tile(const KvReq& r, int rt, const KvAttnParams& p) {
  KvTiles t;
  int i0 = 0, i1 = r.nq - 1, x;
  if (r.R > RT) i0 = rt * RT / p.G, i1 = (imin(r.R, (rt + 1) * RT) - 1) / p.G;
  kv_row_keys(r, i0, p.causal, p.window, &t.lo, &x);
  kv_row_keys(r, i1, p.causal, p.window, &x, &t.hi);
  if (t.hi <= t.lo) {
    t.lo = t.hi = t.t0 = 0;
    t.n = 1;
    return t;
  }
  t.t0 = t.lo / KT;
  t.n = (t.hi + KT - 1) / KT - t.t0;
  return t;
}

template <int RT>
__host__ __device__ __forceinline__ int kv_row_tiles(const KvReq& r) {
  return (r.R + RT - 1) / RT;
}

// Positions of a request on a head's line.
template <int RT, int KT, int COST>
__host__ __device__ __forceinline__ int64_t kv_request_work(const KvReq& r, const KvAttnParams& p) {
  int64_t w = 0;
  const int nt = kv_row_tiles<RT>(r);
#pragma unroll 1
  for (int rt = 0; rt < nt; ++rt) w += kv_row_tile<RT, KT>(r, rt, p).n + COST;
  return w;
}

// First position of part c of C, and the part that holds position x.
__host__ __device__ __forceinline__ int64_t kv_part_begin(int64_t total, int c, int C) {
  if (total <= 0xffffffffll / C) return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(C);
  return total * c / C;
}
__host__ __device__ __forceinline__ int kv_part_of(int64_t total, int64_t x, int C) {
  int c = static_cast<int>((x * C) / total);
  while (c > 0 && kv_part_begin(total, c, C) > x) --c;
  while (c + 1 < C && kv_part_begin(total, c + 1, C) <= x) ++c;
  return c;
}

}  // namespace ab
