// Parameter blocks and launchers of the paged 8-bit cache operators (internal
// to the library).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_kv_cache.h"
#include "common.cuh"

namespace ab {

struct KvTablesParams {
  const int* ctx;
  const int* add;
  int N;
  int* table;
  int64_t table_stride;
  int max_blocks;
  const int* free_blocks;
  int num_free;
  const int* free_start;  // device scalar, or null: 0
  int page_log2, num_blocks, T;
  int* cu;
  int* kv_lens;
  int* slot_map;
  int* positions;
  int* counts;
};

struct KvWriteParams {
  const uint8_t* x[2];  // k, v: 16-bit [T,HKV,D]
  int64_t sx_s[2], sx_h[2];  // element strides
  uint8_t* cache[2];
  int64_t sc_b[2], sc_s[2], sc_h[2];
  float* scale[2];  // [num_blocks, HKV]
  const int* slot_map;
  int T, HKV, D, page_log2, num_blocks;
};

// Attention over the cache.
struct KvAttnParams {
  const uint8_t* q;
  int64_t sq_s, sq_h;  // element strides
  uint8_t* o;
  int64_t so_s, so_h;
  float* lse;
  int64_t sl_s, sl_h;
  const uint8_t* k;
  int64_t sk_b, sk_s, sk_h;
  const uint8_t* v;
  int64_t sv_b, sv_s, sv_h;
  const float* k_scale;
  const float* v_scale;
  const int* table;
  int64_t table_stride;
  int max_blocks, num_blocks, page_log2;
  const int* cu;
  const int* kv_lens;
  int N, T, HQ, HKV, G, D;
  int causal, window;
  int rows_min, rows_max;  // requests of other sizes are left to another kernel
  float scale_log2;        // sm_scale * log2(e), > 0
  // workspace
  int* err;
  int* cta_err;     // per CTA: its error code
  int4* desc;       // per worker: the unit whose split it finishes (see kv_decode.cu)
  float2* part_ml;  // [2 * workers][rows] running max (log2 units) and sum
  float* part_o;    // [2 * workers][rows][D] unnormalised O
  uint64_t timeout_ns;
};

// Tensor maps of the cache's bytes, dims (D, HKV, page_size, num_blocks): box D
// bytes x tokens of one head (a page, but at most a kernel's tile), swizzled over rows of D bytes.
struct KvMaps {
  CUtensorMap k, v;
};

// Requests of at least this many rows (queries * heads of a group) go to the
// prompt kernel, the others to the decode kernel, where both are queued (kv_api.cu).
// 64 requests on 2048 keys, 8 KV heads of 128, decode and prompt kernel: 24 and 32 rows
// 106 us and 143, 48 rows 168 and 145, 64 rows 200 and 149.
constexpr int kKvPrMinRows = 65;

// Decode kernel: keys per tile, and what starting a unit costs in tiles (1 to 4
// tried: each step up to 4 takes 0.3 to 1 % off calls of many units).
constexpr int kKvDecKeys = 32;
constexpr int kKvDecCost = 4;
// Most partial rows of a launch (2 slots a worker, 8 or 16 rows a slot) and most
// workers: these size the workspace and bound the grid.  Units of 16 rows get 256 CTAs
// of the 304 (head dim 128) or 456 (64) that 152 SMs hold.  With rows for all, 64 single
// tokens on 8192 keys, groups of 16, take 65 us instead of 67.5, at head dim 64 47
// instead of 55, 4 drafted tokens, groups of 4, 188 instead of 208, but 6 on 2048 keys
// 111 instead of 106, and the workspace twice its size.
constexpr int kKvDecMaxRows = 32768;
constexpr int kKvDecMaxWorkers = kKvDecMaxRows / 16;

// Prompt kernel: rows of a unit, keys per block, what starting a unit costs in
// blocks, fewest line positions of a CTA's part, most CTAs.
constexpr int kKvPrRows = 256;
constexpr int kKvPrKeys = 128;
constexpr int kKvPrCost = 3;
constexpr int kKvPrMinWork = 5;
constexpr int kKvPrMaxCtas = 160;

cudaError_t launch_kv_tables(const KvTablesParams& p, int grid, cudaStream_t st);
cudaError_t launch_kv_write(const KvWriteParams& p, bool bf16, cudaStream_t st);
// What a kernel leaves to be joined: an error word per CTA, a descriptor per
// worker (``stride`` workers to a part of the line), partial rows of units of
// ``rows`` rows.  workers = 0: nothing.
struct KvJoinPart {
  const int* cta_err;
  const int4* desc;
  const float2* part_ml;
  const float* part_o;
  int workers, ctas, stride, rows;
};
inline KvJoinPart kv_join_part(const KvAttnParams& p, int workers, int ctas, int stride, int rows) {
  return {p.cta_err, p.desc, p.part_ml, p.part_o, workers, ctas, stride, rows};
}

// Both fill ``left`` with what launch_kv_join has to finish.
cudaError_t launch_kv_decode(const KvAttnParams& p, const KvMaps& maps, bool bf16, int sms, KvJoinPart* left,
                             cudaStream_t st);
cudaError_t launch_kv_prompt(const KvAttnParams& p, const KvMaps& maps, bool bf16, int sms, KvJoinPart* left,
                             cudaStream_t st);
// Joins the rows that the kernels of few and of many rows split, and writes the
// call's error word.
cudaError_t launch_kv_join(const KvAttnParams& p, bool bf16, const KvJoinPart& few, const KvJoinPart& many, int sms,
                           cudaStream_t st);

}  // namespace ab
