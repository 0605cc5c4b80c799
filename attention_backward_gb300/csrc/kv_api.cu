// Host entry points of include/attn_kv_cache.h: argument checks, workspace
// layout and launches.  Nothing here allocates memory or keeps state.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn_kv_cache.h"
#include "kernels.h"
#include "kv_cache.h"
#include "kv_launch.h"

namespace {

using namespace ab;

constexpr int64_t kMax32 = int64_t(1) << 31;
// Rows, keys and tokens stay this far below it: the kernels count them in 32 bits,
// up to a few tiles past the last one.
constexpr int64_t kMaxCount = kMax32 - 4096;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Strides in elements of ``bytes`` bytes: positive multiples of 16 bytes.
bool stride_ok(int64_t s, int64_t bytes) { return s > 0 && (s * bytes) % 16 == 0 && s < (int64_t(1) << 40); }

int page_log2(int64_t page_size) {
  return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : page_size == 128 ? 7 : -1;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  return n;
}

attn_status_t launch_status(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH; }

attn_status_t check_cache(const attn_kv_cache_t* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return ATTN_ERR_INVALID_ARG;
  if (c->num_blocks < 1 || c->HKV < 1 || c->page_size < 1 || c->D < 1) return ATTN_ERR_INVALID_ARG;
  if ((c->D != 64 && c->D != 128) || page_log2(c->page_size) < 0) return ATTN_ERR_UNSUPPORTED;
  if (c->HKV > 16384 || c->num_blocks >= kMax32 / c->page_size || c->num_blocks >= kMax32 / c->HKV)
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return ATTN_ERR_INVALID_ARG;
  for (const attn_strides_t* s : {&c->sk, &c->sv})
    if (!stride_ok(s->b, 1) || !stride_ok(s->s, 1) || !stride_ok(s->h, 1)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

bool dtype_ok(attn_dtype_t dt) { return dt == ATTN_DT_F16 || dt == ATTN_DT_BF16; }

bool make_cache_map(CUtensorMap* m, const void* base, const attn_strides_t& st, const attn_kv_cache_t& c,
                    int64_t box_tokens) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.HKV),
                        static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.num_blocks)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(st.h), static_cast<cuuint64_t>(st.s),
                           static_cast<cuuint64_t>(st.b)};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(c.D), 1, static_cast<cuuint32_t>(box_tokens), 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_maps(KvMaps* m, const attn_kv_cache_t& c, int64_t box_tokens) {
  return make_cache_map(&m->k, c.k, c.sk, c, box_tokens) && make_cache_map(&m->v, c.v, c.sv, c, box_tokens);
}

// Workspace of attention over the cache: the header, then for each of its two
// kernels an error word a CTA, a descriptor a worker, and the partial
// rows.
struct KvWs {
  int64_t err_off, desc_off, ml_off, o_off, total;
};

KvWs kv_ws(int64_t start, int64_t workers, int64_t rows, int64_t D) {
  KvWs w;
  w.err_off = start;
  w.desc_off = w.err_off + round_up(workers * 4, 256);
  w.ml_off = w.desc_off + workers * 16;
  w.o_off = w.ml_off + rows * 8;
  w.total = w.o_off + rows * D * 4;
  return w;
}
KvWs kv_ws_decode(int64_t D) { return kv_ws(kHeaderBytes, kKvDecMaxWorkers, kKvDecMaxRows, D); }
KvWs kv_ws_prompt(int64_t D) { return kv_ws(kv_ws_decode(D).total, kKvPrMaxCtas, 2 * kKvPrMaxCtas * kKvPrRows, D); }

// Whether a call of T queries may hold a request of kKvPrMinRows rows or more.
bool kv_may_prompt(int64_t T, int64_t G) { return T * G >= kKvPrMinRows; }

void kv_place(KvAttnParams* p, const KvWs& w, uint8_t* ws) {
  p->cta_err = reinterpret_cast<int*>(ws + w.err_off);
  p->desc = reinterpret_cast<int4*>(ws + w.desc_off);
  p->part_ml = reinterpret_cast<float2*>(ws + w.ml_off);
  p->part_o = reinterpret_cast<float*>(ws + w.o_off);
}

}  // namespace

extern "C" {

attn_status_t attn_kv_block_tables(const int32_t* ctx_lens, const int32_t* new_lens, int64_t num_seqs,
                                   int32_t* block_table, int64_t table_stride, int64_t max_blocks,
                                   const int32_t* free_blocks, int64_t num_free, const int32_t* free_start,
                                   int64_t page_size, int64_t num_blocks, int64_t max_tokens, int32_t* cu_seqlens,
                                   int32_t* kv_lens, int32_t* slot_map, int32_t* positions, int32_t* counts,
                                   void* stream) {
  if (!ctx_lens || !new_lens || !block_table || !cu_seqlens || !kv_lens || !counts) return ATTN_ERR_INVALID_ARG;
  if (num_seqs < 1 || max_blocks < 1 || table_stride < max_blocks || num_free < 0 || num_blocks < 1 ||
      max_tokens < 0 || page_size < 1)
    return ATTN_ERR_INVALID_ARG;
  if ((num_free > 0 && !free_blocks) || (max_tokens > 0 && (!slot_map || !positions))) return ATTN_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(ctx_lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(block_table), static_cast<const void*>(free_blocks),
                        static_cast<const void*>(free_start), static_cast<const void*>(cu_seqlens),
                        static_cast<const void*>(kv_lens), static_cast<const void*>(slot_map),
                        static_cast<const void*>(positions), static_cast<const void*>(counts)})
    if (!aligned(q, 4)) return ATTN_ERR_INVALID_ARG;
  if (kv_lens == ctx_lens || kv_lens == new_lens) return ATTN_ERR_INVALID_ARG;  // every block reads the lengths
  if (page_log2(page_size) < 0) return ATTN_ERR_UNSUPPORTED;
  if (num_seqs > (1 << 20) || max_blocks >= kMax32 / page_size || num_blocks >= kMax32 / page_size ||
      num_free >= kMax32 || max_tokens >= kMax32)
    return ATTN_ERR_UNSUPPORTED;
  KvTablesParams p{};
  p.ctx = ctx_lens, p.add = new_lens, p.N = static_cast<int>(num_seqs);
  p.table = block_table, p.table_stride = table_stride, p.max_blocks = static_cast<int>(max_blocks);
  p.free_blocks = free_blocks, p.num_free = static_cast<int>(num_free), p.free_start = free_start;
  p.page_log2 = page_log2(page_size), p.num_blocks = static_cast<int>(num_blocks);
  p.T = static_cast<int>(max_tokens);
  p.cu = cu_seqlens, p.kv_lens = kv_lens, p.slot_map = slot_map, p.positions = positions, p.counts = counts;
  return launch_status(launch_kv_tables(p, sm_count(), static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_kv_cache_write(const void* k, attn_strides_t sk, const void* v, attn_strides_t sv,
                                  const int32_t* slot_map, int64_t T, attn_dtype_t dtype,
                                  const attn_kv_cache_t* cache, void* stream) {
  if (const attn_status_t st = check_cache(cache); st != ATTN_OK) return st;
  if (T < 0) return ATTN_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || T > kMaxCount) return ATTN_ERR_UNSUPPORTED;
  if (T == 0) return ATTN_OK;
  if (!k || !v || !slot_map) return ATTN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 4)) return ATTN_ERR_INVALID_ARG;
  for (const attn_strides_t* s : {&sk, &sv})
    if (!stride_ok(s->s, 2) || !stride_ok(s->h, 2)) return ATTN_ERR_INVALID_ARG;
  KvWriteParams p{};
  p.x[0] = static_cast<const uint8_t*>(k), p.x[1] = static_cast<const uint8_t*>(v);
  p.sx_s[0] = sk.s, p.sx_h[0] = sk.h, p.sx_s[1] = sv.s, p.sx_h[1] = sv.h;
  p.cache[0] = static_cast<uint8_t*>(cache->k), p.cache[1] = static_cast<uint8_t*>(cache->v);
  p.sc_b[0] = cache->sk.b, p.sc_s[0] = cache->sk.s, p.sc_h[0] = cache->sk.h;
  p.sc_b[1] = cache->sv.b, p.sc_s[1] = cache->sv.s, p.sc_h[1] = cache->sv.h;
  p.scale[0] = cache->k_scale, p.scale[1] = cache->v_scale;
  p.slot_map = slot_map;
  p.T = static_cast<int>(T), p.HKV = static_cast<int>(cache->HKV), p.D = static_cast<int>(cache->D);
  p.page_log2 = page_log2(cache->page_size), p.num_blocks = static_cast<int>(cache->num_blocks);
  return launch_status(launch_kv_write(p, dtype == ATTN_DT_BF16, static_cast<cudaStream_t>(stream)));
}

size_t attn_fwd_kv_cache_workspace_size(int64_t T, int64_t HQ, int64_t HKV, int64_t D) {
  if (T < 0 || HQ < 1 || HKV < 1 || HQ % HKV || (D != 64 && D != 128) || T > kMaxCount / HQ) return 0;
  return static_cast<size_t>(kv_may_prompt(T, HQ / HKV) ? kv_ws_prompt(D).total : kv_ws_decode(D).total);
}

attn_status_t attn_fwd_kv_cache(const void* q, attn_strides_t sq, int64_t T, int64_t HQ, attn_dtype_t dtype,
                                float sm_scale, const attn_kv_cache_t* cache, const int32_t* block_table,
                                int64_t table_stride, int64_t max_blocks, const int32_t* cu_seqlens,
                                const int32_t* kv_lens, int64_t num_seqs, int32_t causal, int32_t window_left, void* o,
                                attn_strides_t so, float* lse, attn_strides_t slse, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (const attn_status_t st = check_cache(cache); st != ATTN_OK) return st;
  if (T < 0 || HQ < 1 || HQ % cache->HKV != 0 || num_seqs < 1 || max_blocks < 1 || table_stride < max_blocks)
    return ATTN_ERR_INVALID_ARG;
  if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return ATTN_ERR_INVALID_ARG;
  if (window_left == 0 || window_left < -1) return ATTN_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || T > kMaxCount / HQ || num_seqs > (1 << 20) || max_blocks > kMaxCount / cache->page_size)
    return ATTN_ERR_UNSUPPORTED;
  if (T == 0) return ATTN_OK;
  if (!q || !o || !lse || !block_table || !cu_seqlens || !kv_lens || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(workspace, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
      !aligned(cu_seqlens, 4) || !aligned(kv_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  for (const attn_strides_t* s : {&sq, &so})
    if (!stride_ok(s->s, 2) || !stride_ok(s->h, 2)) return ATTN_ERR_INVALID_ARG;
  if (slse.s < 1 || slse.h < 1) return ATTN_ERR_INVALID_ARG;
  if (workspace_bytes < attn_fwd_kv_cache_workspace_size(T, HQ, cache->HKV, cache->D)) return ATTN_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  KvAttnParams p{};
  p.q = static_cast<const uint8_t*>(q), p.sq_s = sq.s, p.sq_h = sq.h;
  p.o = static_cast<uint8_t*>(o), p.so_s = so.s, p.so_h = so.h;
  p.lse = lse, p.sl_s = slse.s, p.sl_h = slse.h;
  p.k = static_cast<const uint8_t*>(cache->k), p.sk_b = cache->sk.b, p.sk_s = cache->sk.s, p.sk_h = cache->sk.h;
  p.v = static_cast<const uint8_t*>(cache->v), p.sv_b = cache->sv.b, p.sv_s = cache->sv.s, p.sv_h = cache->sv.h;
  p.k_scale = cache->k_scale, p.v_scale = cache->v_scale;
  p.table = block_table, p.table_stride = table_stride, p.max_blocks = static_cast<int>(max_blocks);
  p.num_blocks = static_cast<int>(cache->num_blocks), p.page_log2 = page_log2(cache->page_size);
  p.cu = cu_seqlens, p.kv_lens = kv_lens, p.N = static_cast<int>(num_seqs), p.T = static_cast<int>(T);
  p.HQ = static_cast<int>(HQ), p.HKV = static_cast<int>(cache->HKV), p.G = static_cast<int>(HQ / cache->HKV);
  p.D = static_cast<int>(cache->D);
  p.causal = causal ? 1 : 0, p.window = window_left;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.err = &reinterpret_cast<WsHeader*>(ws)->err;
  p.timeout_ns = kWaitTimeoutNs;
  const bool bf16 = dtype == ATTN_DT_BF16;
  const int sms = sm_count();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Which kernels: where both are queued, requests of kKvPrMinRows rows or more go to
  // the prompt kernel, the others to the decode kernel.  Either serves any number of
  // rows, and one of them takes all where the mean of rows a request (the host knows
  // no more) is below a quarter of that limit or, for several requests, from four times
  // it on.  A prompt kernel that finds nothing costs 5 us (32 requests of 6 tokens, one
  // head a group: 96 us, 101 with it).  What the rule costs is a request far from the
  // mean: 256 tokens beside a chunk of 512, groups of 4, mean 12: 433 us, 267 with
  // both kernels; 160 beside 2048, groups of 1, mean 14: 1085 and 606; 1024 beside
  // 14000, 4 heads, mean 15: 1566 and 334; 8 tokens of 65536 keys beside a chunk of 4096,
  // groups of 4, mean 1824: 668 and 404.
  const int64_t mean = T * p.G / num_seqs;
  const bool prompts = kv_may_prompt(T, p.G) && mean >= kKvPrMinRows / 4;
  const bool decodes = !prompts || (num_seqs > 1 && mean < 4 * kKvPrMinRows);
  KvMaps small, large;
  if ((decodes && !make_maps(&small, *cache, std::min<int64_t>(cache->page_size, kKvDecKeys))) ||
      (prompts && !make_maps(&large, *cache, std::min<int64_t>(cache->page_size, kKvPrKeys))))
    return ATTN_ERR_INVALID_ARG;
  p.rows_min = 0, p.rows_max = prompts ? kKvPrMinRows - 1 : 0x7fffffff;
  KvJoinPart few{}, many{};
  if (decodes) {
    kv_place(&p, kv_ws_decode(cache->D), ws);
    if (const cudaError_t e = launch_kv_decode(p, small, bf16, sms, &few, st); e != cudaSuccess) return launch_status(e);
  }
  if (prompts) {
    p.rows_min = decodes ? kKvPrMinRows : 0, p.rows_max = 0x7fffffff;
    kv_place(&p, kv_ws_prompt(cache->D), ws);
    if (const cudaError_t e = launch_kv_prompt(p, large, bf16, sms, &many, st); e != cudaSuccess)
      return launch_status(e);
  }
  return launch_status(launch_kv_join(p, bf16, few, many, sms, st));
}

}  // extern "C"
