// Host entry points of include/attn_rope.h and include/attn_latent.h: argument
// checks, workspace layout and launches.  Nothing here allocates memory or keeps
// state.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn_latent.h"
#include "attn_rope.h"
#include "common.cuh"
#include "kv_launch.h"
#include "latent.h"
#include "rope.h"

namespace {

using namespace ab;

constexpr int64_t kMax32 = int64_t(1) << 31;
constexpr int64_t kRopeMaxHeads = 1 << 20;
constexpr int64_t kMaxCount = kMax32 - 4096;  // rows and tokens are counted in 32 bits, up to a few tiles past the last

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Stride in 16-bit elements: a positive multiple of 16 bytes.
bool stride_ok(int64_t s) { return s > 0 && s % 8 == 0 && s < (int64_t(1) << 39); }

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

bool dtype_ok(attn_dtype_t dt) { return dt == ATTN_DT_F16 || dt == ATTN_DT_BF16; }

// A 4-D tensor of 16-bit values, 128-byte swizzle; ``strides`` (elements) and
// ``box`` of the dimensions after the first, whose box is 64 columns.
bool make_map(CUtensorMap* m, const void* base, attn_dtype_t dt, int64_t D, const int64_t (&size)[3],
              const int64_t (&stride)[3], const int (&rows)[3]) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D)}, strides[3];
  cuuint32_t box[4] = {64}, es[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = static_cast<cuuint64_t>(size[i]), strides[i] = static_cast<cuuint64_t>(stride[i] * 2);
    box[i + 1] = static_cast<cuuint32_t>(rows[i]);
  }
  return fn(m, dt == ATTN_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [B,S,H,D], box 64 columns x ``heads`` x ``rows`` of the sequence.
bool make_bshd_map(CUtensorMap* m, const void* base, attn_dtype_t dt, int64_t B, int64_t S, int64_t H, int64_t D,
                   const attn_strides_t& st, int heads, int rows) {
  return make_map(m, base, dt, D, {H, S, B}, {st.h, st.s, st.b}, {heads, rows, 1});
}

attn_status_t check_rope(const attn_rope_tensor_t* t, int64_t R) {
  if (!t->x || !t->y || t->H < 1 || t->D < 1 || t->start < 0) return ATTN_ERR_INVALID_ARG;
  if (t->D % 8 || t->start % 8 || t->start > t->D - R) return ATTN_ERR_INVALID_ARG;
  if (t->D > 1024) return ATTN_ERR_UNSUPPORTED;
  if (!aligned(t->x, 16) || !aligned(t->y, 16)) return ATTN_ERR_INVALID_ARG;
  for (const attn_strides_t* s : {&t->sx, &t->sy})
    if (!stride_ok(s->b) || !stride_ok(s->s) || !stride_ok(s->h)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

RopeTensor rope_tensor(const attn_rope_tensor_t& t, int64_t R) {
  const bool in_place = t.x == t.y && t.sx.b == t.sy.b && t.sx.s == t.sy.s && t.sx.h == t.sy.h;
  return {static_cast<const uint8_t*>(t.x), t.sx.b, t.sx.s, t.sx.h, static_cast<uint8_t*>(t.y), t.sy.b, t.sy.s, t.sy.h,
          static_cast<int>(t.H), static_cast<int>(t.start), in_place ? 0 : static_cast<int>(t.D - R) / 8};
}

attn_status_t check_cache(const attn_latent_cache_t* c) {
  if (!c || !c->rows || c->num_blocks < 1 || c->page_size < 1) return ATTN_ERR_INVALID_ARG;
  if (page_log2(c->page_size) < 0 || c->num_blocks >= kMax32 / c->page_size) return ATTN_ERR_UNSUPPORTED;
  if (!aligned(c->rows, 16) || !stride_ok(c->row_stride) || c->row_stride < kLatRow) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// Workspace of attention over the cache: the header, an error word and a
// descriptor a CTA, then two slots of partial rows a CTA.
struct LatWs {
  int64_t err_off, desc_off, ml_off, o_off, total;
};
LatWs lat_ws() {
  LatWs w;
  w.err_off = kHeaderBytes;
  w.desc_off = w.err_off + round_up(kLatMaxCtas * 4, 256);
  w.ml_off = w.desc_off + kLatMaxCtas * 16;
  w.o_off = w.ml_off + 2 * kLatMaxCtas * kLatRows * 8;
  w.total = w.o_off + int64_t(2) * kLatMaxCtas * kLatRows * kLatDim * 4;
  return w;
}

// Pairs of 128-row query tiles of the expanded form; a packed batch may add one a sequence.
int64_t fwd_pairs(int64_t B, int64_t S, int64_t H, int64_t num_seqs) { return ((S + 255) / 256 + num_seqs) * B * H; }

// Partial rows of lists that are split, a slot a CTA.
constexpr int64_t kListPartBytes = int64_t(kLatMaxCtas) * kLatRows * (8 + kLatDim * 4);

}  // namespace

extern "C" {

attn_status_t attn_rope(const attn_rope_tensor_t* q, const attn_rope_tensor_t* k, int64_t B, int64_t S,
                        attn_dtype_t dtype, const int32_t* positions, int64_t positions_b, const uint64_t* steps,
                        int64_t rotary_dim, float scale, int32_t interleaved, int32_t inverse, void* stream) {
  if (!q || B < 1 || S < 0 || rotary_dim < 1 || positions_b < 0 || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (rotary_dim % 16 || rotary_dim > 1024 || !dtype_ok(dtype)) return ATTN_ERR_UNSUPPORTED;
  if (S == 0) return ATTN_OK;
  if (const attn_status_t st = check_rope(q, rotary_dim); st != ATTN_OK) return st;
  if (k)
    if (const attn_status_t st = check_rope(k, rotary_dim); st != ATTN_OK) return st;
  // (threads of a token are counted in 32 bits too)
  if (q->H > kRopeMaxHeads || (k && k->H > kRopeMaxHeads) || B > kMaxCount) return ATTN_ERR_UNSUPPORTED;
  const int64_t heads = q->H + (k ? k->H : 0);
  if (heads > kRopeMaxHeads || S > kMaxCount / B || heads > kMaxCount / (B * S))
    return ATTN_ERR_UNSUPPORTED;
  if (!positions || !steps || !aligned(positions, 4) || !aligned(steps, 8)) return ATTN_ERR_INVALID_ARG;
  RopeParams p{};
  p.t[0] = rope_tensor(*q, rotary_dim);
  if (k) p.t[1] = rope_tensor(*k, rotary_dim);
  p.heads = static_cast<int>(heads);
  p.B = static_cast<int>(B), p.S = static_cast<int>(S), p.R = static_cast<int>(rotary_dim);
  p.pos = positions, p.pos_b = positions_b, p.steps = steps, p.scale = scale;
  p.inter = interleaved ? 1 : 0, p.inverse = inverse ? 1 : 0;
  return launch_status(launch_rope(p, dtype == ATTN_DT_BF16, sm_count(), static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_latent_cache_write(const void* kv, int64_t kv_stride, const int32_t* slot_map, int64_t T,
                                      attn_dtype_t dtype, const void* norm_weight, float norm_eps,
                                      const int32_t* positions, const uint64_t* steps, float rope_scale,
                                      int32_t interleaved, const attn_latent_cache_t* cache, void* out,
                                      int64_t out_stride, void* stream) {
  if (const attn_status_t st = check_cache(cache); st != ATTN_OK) return st;
  if (T < 0 || (positions == nullptr) != (steps == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (norm_weight && (!(norm_eps >= 0.f) || !std::isfinite(norm_eps) || !aligned(norm_weight, 16))) return ATTN_ERR_INVALID_ARG;
  if (steps && (!std::isfinite(rope_scale) || !aligned(steps, 8) || !aligned(positions, 4))) return ATTN_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || T > kMaxCount) return ATTN_ERR_UNSUPPORTED;
  if (T == 0) return ATTN_OK;
  if (!kv || !slot_map || !aligned(kv, 16) || !aligned(slot_map, 4) || !stride_ok(kv_stride) || kv_stride < kLatRow)
    return ATTN_ERR_INVALID_ARG;
  if (out && (!aligned(out, 16) || !stride_ok(out_stride) || out_stride < kLatRow || (out == kv && out_stride != kv_stride)))
    return ATTN_ERR_INVALID_ARG;
  LatWriteParams p{};
  p.kv = static_cast<const uint8_t*>(kv), p.kv_stride = kv_stride;
  p.cache = static_cast<uint8_t*>(cache->rows), p.row_stride = cache->row_stride;
  p.out = static_cast<uint8_t*>(out), p.out_stride = out_stride;
  p.slot_map = slot_map, p.weight = static_cast<const uint8_t*>(norm_weight), p.eps = norm_eps;
  p.pos = positions, p.steps = steps, p.scale = rope_scale, p.inter = interleaved ? 1 : 0;
  p.T = static_cast<int>(T), p.slots = static_cast<int>(cache->num_blocks * cache->page_size);
  return launch_status(launch_latent_write(p, dtype == ATTN_DT_BF16, static_cast<cudaStream_t>(stream)));
}

size_t attn_fwd_latent_cache_workspace_size(void) { return static_cast<size_t>(lat_ws().total); }

attn_status_t attn_fwd_latent_cache(const void* q, attn_strides_t sq, int64_t T, int64_t H, attn_dtype_t dtype,
                                    float sm_scale, const attn_latent_cache_t* cache, const int32_t* block_table,
                                    int64_t table_stride, int64_t max_blocks, const int32_t* cu_seqlens,
                                    const int32_t* kv_lens, int64_t num_seqs, int32_t causal, void* o,
                                    attn_strides_t so, float* lse, attn_strides_t slse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  if (const attn_status_t st = check_cache(cache); st != ATTN_OK) return st;
  if (T < 0 || H < 1 || num_seqs < 1 || max_blocks < 1 || table_stride < max_blocks) return ATTN_ERR_INVALID_ARG;
  if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return ATTN_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || T > kMaxCount / H || H > kMaxCount || num_seqs > (1 << 20) ||
      max_blocks > kMaxCount / cache->page_size)
    return ATTN_ERR_UNSUPPORTED;
  if (T == 0) return ATTN_OK;
  if (!q || !o || !lse || !block_table || !cu_seqlens || !kv_lens || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(workspace, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
      !aligned(cu_seqlens, 4) || !aligned(kv_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  for (const attn_strides_t* s : {&sq, &so})
    if (!stride_ok(s->s) || !stride_ok(s->h)) return ATTN_ERR_INVALID_ARG;
  if (slse.s < 1 || slse.h < 1) return ATTN_ERR_INVALID_ARG;
  const LatWs w = lat_ws();
  if (workspace_bytes < static_cast<size_t>(w.total)) return ATTN_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  LatParams lp{};
  KvAttnParams& p = lp.a;
  // Rows of q that are evenly spaced come as boxes of 64, others (heads of a wider tensor) by
  // copies of one warp: 1.0 and 6 us a unit of 64 rows.
  CUtensorMap rows{};
  if (H == 1 || T == 1 || sq.s == H * sq.h) {
    const int64_t step = H == 1 ? sq.s : sq.h;
    if (!make_map(&rows, q, dtype, kLatRow, {T * H, 1, 1}, {step, step, step}, {kLatRows, 1, 1})) return ATTN_ERR_INVALID_ARG;
  } else {
    p.q = static_cast<const uint8_t*>(q), p.sq_s = sq.s, p.sq_h = sq.h;
  }
  p.o = static_cast<uint8_t*>(o), p.so_s = so.s, p.so_h = so.h;
  p.lse = lse, p.sl_s = slse.s, p.sl_h = slse.h;
  lp.rows = static_cast<const uint8_t*>(cache->rows), lp.row_stride = cache->row_stride;
  p.table = block_table, p.table_stride = table_stride, p.max_blocks = static_cast<int>(max_blocks);
  p.num_blocks = static_cast<int>(cache->num_blocks), p.page_log2 = page_log2(cache->page_size);
  p.cu = cu_seqlens, p.kv_lens = kv_lens, p.N = static_cast<int>(num_seqs), p.T = static_cast<int>(T);
  p.HQ = p.G = static_cast<int>(H), p.HKV = 1;
  p.causal = causal ? 1 : 0, p.window = -1, p.rows_min = 0, p.rows_max = 0x7fffffff;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.err = &reinterpret_cast<WsHeader*>(ws)->err;
  p.cta_err = reinterpret_cast<int*>(ws + w.err_off);
  p.desc = reinterpret_cast<int4*>(ws + w.desc_off);
  p.part_ml = reinterpret_cast<float2*>(ws + w.ml_off);
  p.part_o = reinterpret_cast<float*>(ws + w.o_off);
  p.timeout_ns = kWaitTimeoutNs;
  const bool bf16 = dtype == ATTN_DT_BF16;
  const int sms = sm_count();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // CTAs that share their keys: two where the mean of rows a request (the host knows no
  // more) does not fit one.
  const int group = T * H > num_seqs * kLatRows ? 2 : 1;
  const int ctas = imin(sms, kLatMaxCtas) / group * group;
  if (const cudaError_t e = launch_latent_cache(lp, rows, bf16, group, sms, st); e != cudaSuccess) return launch_status(e);
  return launch_status(launch_latent_join(lp, bf16, group, ctas, sms, st));
}

size_t attn_fwd_sparse_workspace_size(int64_t B, int64_t S, int64_t HKV) {
  if (B < 1 || S < 1 || HKV < 1 || B >= kMax32 || HKV >= kMax32 || B > kMaxCount / HKV || B * HKV > kMaxCount / S) return 0;
  return static_cast<size_t>(kHeaderBytes + (2 * B * S * HKV <= kLatMaxCtas ? kListPartBytes : 0));
}

attn_status_t attn_fwd_sparse(const void* q, attn_strides_t sq, const void* kv, attn_strides_t skv, const int32_t* idx,
                              attn_strides_t sidx, int64_t B, int64_t S, int64_t SKV, int64_t H, int64_t HKV,
                              int64_t DQK, int64_t DV, int64_t topk, attn_dtype_t dtype, float sm_scale, void* o,
                              attn_strides_t so, float* lse, attn_strides_t slse, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!q || !kv || !idx || !o || !lse || !workspace) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || S < 1 || SKV < 1 || H < 1 || HKV < 1 || H % HKV != 0 || topk < 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale) || !(sm_scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (DQK != kLatRow || DV != kLatDim || H / HKV > kLatRows || !dtype_ok(dtype)) return ATTN_ERR_UNSUPPORTED;
  if (B >= kMax32 || HKV >= kMax32 || S >= kMax32 || SKV >= kMax32 || B > kMaxCount / HKV ||
      B * HKV > kMaxCount / S || B * HKV > kMaxCount / SKV || topk > kMaxCount)
    return ATTN_ERR_UNSUPPORTED;
  for (const void* x : {q, kv, static_cast<const void*>(o), static_cast<const void*>(workspace)})
    if (!aligned(x, 16)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(idx, 4) || !aligned(lse, 4)) return ATTN_ERR_INVALID_ARG;
  for (const attn_strides_t* s : {&sq, &so})
    if (!stride_ok(s->b) || !stride_ok(s->s) || !stride_ok(s->h)) return ATTN_ERR_INVALID_ARG;
  // the rows are gathered as those of a [B*SKV*HKV, 576] matrix
  if (skv.h < kLatRow || skv.h % 8 || skv.s != HKV * skv.h || skv.b != SKV * skv.s) return ATTN_ERR_UNSUPPORTED;
  if (sidx.b < 0 || sidx.s < 0 || sidx.h < 0 || slse.b < 0 || slse.s < 0 || slse.h < 0) return ATTN_ERR_INVALID_ARG;
  if (workspace_bytes < static_cast<size_t>(kHeaderBytes)) return ATTN_ERR_WORKSPACE;
  CUtensorMap heads;
  if (!make_bshd_map(&heads, q, dtype, B, S, H, kLatRow, sq, kLatRows, 1)) return ATTN_ERR_INVALID_ARG;
  LatParams lp{};
  KvAttnParams& p = lp.a;
  lp.rows = static_cast<const uint8_t*>(kv), lp.row_stride = skv.h;
  p.o = static_cast<uint8_t*>(o), p.so_s = so.s, p.so_h = so.h, lp.so_b = so.b;
  p.lse = lse, p.sl_s = slse.s, p.sl_h = slse.h, lp.sl_b = slse.b;
  lp.idx = idx, lp.si_b = sidx.b, lp.si_s = sidx.s, lp.si_h = sidx.h;
  lp.B = static_cast<int>(B), lp.S = static_cast<int>(S), lp.SKV = static_cast<int>(SKV);
  lp.HKV = static_cast<int>(HKV), lp.gh = static_cast<int>(H / HKV), lp.topk = static_cast<int>(topk);
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.err = &static_cast<WsHeader*>(workspace)->err;
  p.timeout_ns = kWaitTimeoutNs;
  const int sms = imin(sm_count(), kLatMaxCtas);
  // Lists that leave CTAs idle are split over them, two tiles a part at least, where the
  // workspace has room for the parts.  64 heads, 2048 rows a list: 48 us whole, 13.3 for
  // one token in 16 parts, 22.5 for 32 in 4, 35 for 76 in 2.
  lp.splits = 1;
  if (workspace_bytes >= static_cast<size_t>(kHeaderBytes + kListPartBytes)) {
    lp.splits = static_cast<int>(std::max<int64_t>(1, std::min(sms / (B * S * HKV), (topk + 2 * kLatKeys - 1) / (2 * kLatKeys))));
    p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + kHeaderBytes);
    p.part_o = reinterpret_cast<float*>(p.part_ml + kLatMaxCtas * kLatRows);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_status(launch_latent_lists(lp, heads, dtype == ATTN_DT_BF16, sms, st));
}

size_t attn_fwd_latent_workspace_size(int64_t B, int64_t S, int64_t H, int64_t num_seqs) {
  if (B < 1 || S < 1 || H < 1 || num_seqs < 0 || num_seqs > (1 << 20) || B > 65535 || H > 65535 || S > kMaxCount / (B * H))
    return 0;
  const int64_t parts = num_seqs == 0 || 2 * fwd_pairs(B, S, H, num_seqs) <= kLatFwdMaxUnits ? kLatFwdMaxUnits * kLatFwdRows : 0;
  return static_cast<size_t>(kHeaderBytes + parts * (8 + 128 * 4));
}

attn_status_t attn_fwd_latent(const void* q, attn_strides_t sq, const void* kn, attn_strides_t skn, const void* kr,
                              attn_strides_t skr, const void* v, attn_strides_t sv, int64_t B, int64_t S, int64_t H,
                              attn_dtype_t dtype, float sm_scale, const attn_mask_t* mask, void* o, attn_strides_t so,
                              float* lse, attn_strides_t slse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !kn || !kr || !v || !o || !lse || !workspace) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || S < 1 || H < 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale) || !(sm_scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (!dtype_ok(dtype)) return ATTN_ERR_UNSUPPORTED;
  for (const void* x : {q, kn, kr, v, static_cast<const void*>(o), static_cast<const void*>(workspace)})
    if (!aligned(x, 16)) return ATTN_ERR_INVALID_ARG;
  for (const attn_strides_t* st : {&sq, &skn, &sv, &so})
    if (!stride_ok(st->b) || !stride_ok(st->s) || !stride_ok(st->h)) return ATTN_ERR_INVALID_ARG;
  if (!stride_ok(skr.b) || !stride_ok(skr.s)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || slse.b < 0 || slse.s < 0 || slse.h < 0) return ATTN_ERR_INVALID_ARG;
  int64_t Sk = S;
  LatFwdParams p{};
  if (mask) {
    if (mask->window_left == 0 || mask->window_left < -1) return ATTN_ERR_INVALID_ARG;
    if (mask->window_left > 0) return ATTN_ERR_UNSUPPORTED;
    p.causal = mask->causal ? 1 : 0;
    p.cu_seqlens = mask->cu_seqlens;
    if (p.cu_seqlens) {
      if (B != 1 || mask->num_seqs < 1 || mask->num_seqs > (1 << 20) || !aligned(p.cu_seqlens, 4)) return ATTN_ERR_INVALID_ARG;
      p.num_seqs = mask->num_seqs;
    }
    if (mask->kv_len < 0 || (p.cu_seqlens && mask->kv_len != 0 && mask->kv_len != S)) return ATTN_ERR_INVALID_ARG;
    if (mask->kv_len > 0) Sk = mask->kv_len;
  }
  if (B > 65535 || H > 65535 || S > kMaxCount / (B * H) || Sk > kMaxCount / (B * H)) return ATTN_ERR_UNSUPPORTED;
  const int64_t pairs = fwd_pairs(B, S, H, p.num_seqs);
  if (pairs > kMaxCount) return ATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < attn_fwd_latent_workspace_size(B, S, H, p.num_seqs)) return ATTN_ERR_WORKSPACE;
  LatFwdMaps m;
  if (!make_bshd_map(&m.q, q, dtype, B, S, H, 192, sq, 1, 128) ||
      !make_bshd_map(&m.kn, kn, dtype, B, Sk, H, 128, skn, 1, 128) ||
      !make_bshd_map(&m.kr, kr, dtype, B, Sk, 1, 64, {skr.b, skr.s, 64}, 1, 128) ||
      !make_bshd_map(&m.v, v, dtype, B, Sk, H, 128, sv, 1, 128))
    return ATTN_ERR_INVALID_ARG;
  p.B = static_cast<int>(B), p.S = static_cast<int>(S), p.Sk = static_cast<int>(Sk), p.H = static_cast<int>(H);
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.o = static_cast<uint8_t*>(o), p.so_b = so.b, p.so_s = so.s, p.so_h = so.h;
  p.lse = lse, p.sl_b = slse.b, p.sl_s = slse.s, p.sl_h = slse.h;
  p.err = &static_cast<WsHeader*>(workspace)->err;
  p.unit_counter = &static_cast<WsHeader*>(workspace)->tile_counter;
  p.timeout_ns = kWaitTimeoutNs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int sms = imin(sm_count(), kLatFwdMaxUnits);
  // Pairs that leave CTAs idle, those of the last round over the CTAs, are split over them,
  // two key blocks a part at least, where one sees 1024 keys (2048 behind whole rounds): 8
  // queries on 8192 keys, one head 128 -> 19 us, 300 on 4000, 8 heads 66 -> 23, 1024 on 1024,
  // 8 heads 20.3 -> 18.7, 2048 on 8192, 64 heads 431 -> 405; 512 on 512, 16 heads would take
  // 17.8 instead of 13.5, 8192 on 8192, 16 heads, whose last pairs see 1024, 239 instead of 231.
  // (Of a packed batch the host has only a bound of the pairs.)
  p.splits = 1, p.whole = 0x7fffffff;
  const int64_t last = p.cu_seqlens ? (pairs < sms ? pairs : 0) : pairs % sms;
  if (last > 0) {
    const int64_t rows = (last + B * H - 1) / (B * H) * kLatFwdRows;
    const int64_t keys = p.causal && !p.cu_seqlens ? std::min(Sk, std::max<int64_t>(0, Sk - S + rows)) : Sk;
    p.splits = keys < (pairs < sms ? 1024 : 2048) ? 1 : static_cast<int>(std::min(sms / last, (keys + 255) / 256));
  }
  const int64_t split = p.splits > 1 ? last : 0, units = pairs - split + split * p.splits;
  if (split > 0) {
    p.whole = static_cast<int>(pairs - split);
    p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + kHeaderBytes);
    p.part_o = reinterpret_cast<float*>(p.part_ml + kLatFwdMaxUnits * kLatFwdRows);
  }
  p.units = static_cast<int>(units);
  // the counter of units starts clear where some are drawn (without, 128 on 128, 4 heads 10.3
  // -> 7.0 us)
  if (units > sms && cudaMemsetAsync(workspace, 0, kHeaderBytes, st) != cudaSuccess) return ATTN_ERR_LAUNCH;
  return launch_status(launch_latent_fwd(p, m, dtype == ATTN_DT_BF16, static_cast<int>(split),
                                         static_cast<int>(units < sms ? units : sms), st));
}

}  // extern "C"
