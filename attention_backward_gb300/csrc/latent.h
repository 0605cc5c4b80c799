// Parameter blocks and launchers of latent attention (internal to the library).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_latent.h"
#include "kv_cache.h"

namespace ab {

constexpr int kLatRow = ATTN_LATENT_ROW, kLatDim = ATTN_LATENT_DIM, kLatRot = kLatRow - kLatDim;

struct LatWriteParams {
  const uint8_t* kv;
  int64_t kv_stride;  // elements
  uint8_t* cache;
  int64_t row_stride;
  uint8_t* out;  // null: none
  int64_t out_stride;
  const int* slot_map;
  const uint8_t* weight;  // 16-bit [512], or null
  float eps;
  const int* pos;
  const uint64_t* steps;  // null: not turned
  float scale;
  int inter, T;
  int slots;  // num_blocks * page_size
};

cudaError_t launch_latent_write(const LatWriteParams& p, bool bf16, cudaStream_t st);

// Attention over latent rows.  Over the cache: requests as kv_sched.cuh reads
// them from ``a`` (HKV = 1, G = H).  Over lists: ``a`` holds q, o, lse, scale and error
// word, with batch strides and lists here.
struct LatParams {
  KvAttnParams a;
  const uint8_t* rows;  // of the cache, or kv
  int64_t row_stride;   // elements
  // lists
  const int* idx;
  int64_t si_b, si_s, si_h;
  int64_t so_b, sl_b;
  int B, S, SKV, HKV, gh, topk;
  int splits;  // parts of a list's tiles, a CTA each (1: whole)
};

// Unit u of the lists' line: later tokens first, whose lists are longest as a rule.
struct LatListUnit {
  int b, t, g;
};
__host__ __device__ inline LatListUnit list_unit(int u, const LatParams& p) {
  const int n = p.B * p.HKV, bg = u % n;
  return {bg / p.HKV, p.S - 1 - u / n, bg % p.HKV};
}

// Rows (query, head) of a CTA, keys a tile, what starting a unit costs in tiles,
// fewest line positions of a part, most CTAs.
constexpr int kLatRows = 64;
constexpr int kLatKeys = 64;
constexpr int kLatCost = 2;
constexpr int kLatMinWork = 2;
constexpr int kLatMaxCtas = 160;

// A weight is 2^((score - reference) scale_log2 + kLatTop); partial rows hold the reference and
// the weights' sum.
constexpr float kLatTop = 7.f;

// ``group``: CTAs (1 or 2) that share a part of the line, 64 rows each of its units.
// ``q``: where a.q is null, rows of q as dims (576, T * H, 1, 1), box 64 columns x 64 rows.
cudaError_t launch_latent_cache(const LatParams& p, const CUtensorMap& q, bool bf16, int group, int sms,
                                cudaStream_t st);
// ``q``: dims (576, H, S, B), box 64 columns x 64 heads of a token.
cudaError_t launch_latent_lists(const LatParams& p, const CUtensorMap& q, bool bf16, int sms, cudaStream_t st);
// Joins rows that were split over CTAs and, of the cache (group > 0), writes the call's error word.
cudaError_t launch_latent_join(const LatParams& p, bool bf16, int group, int ctas, int sms, cudaStream_t st);

// The expanded form: most parts of pairs of query tiles, and their rows.
constexpr int kLatFwdMaxUnits = 160;
constexpr int kLatFwdRows = 256;
struct LatFwdParams {
  int B, S, Sk, H;
  int causal;
  const int* cu_seqlens;
  int num_seqs;
  float scale_log2;
  uint8_t* o;
  int64_t so_b, so_s, so_h;
  float* lse;
  int64_t sl_b, sl_s, sl_h;
  int* err;
  int* unit_counter;
  int units;
  uint64_t timeout_ns;
  int whole;        // pairs of query tiles that are a unit each (2^31 - 1: all)
  int splits;       // units of each further pair, of a share of its key blocks each
  float2* part_ml;  // [parts][256 rows] reference (a score) and sum
  float* part_o;    // [parts][256 rows][128]
};
struct LatFwdMaps {
  CUtensorMap q, kn, kr, v;  // box 64 columns x 128 rows of one head
};
// ``split_pairs``: at least the pairs of query tiles from p.whole on, 0 where none is split.
cudaError_t launch_latent_fwd(const LatFwdParams& p, const LatFwdMaps& m, bool bf16, int split_pairs, int grid, cudaStream_t st);

}  // namespace ab
