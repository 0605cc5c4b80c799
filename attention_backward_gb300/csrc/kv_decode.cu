// Attention over the paged 8-bit cache for few rows (query, head of the group)
// per KV head: single tokens, drafted tokens.
//
//   x_ij = sm_scale log2(e) ks[page j] (q_i . k_j),  p_ij = 2^(x_ij - m_i)
//   O_i  = sum_j p_ij vs[page j] v_j / l_i,  l_i = sum_j p_ij,
//   LSE_i = (m_i + log2 l_i) ln 2
//
// with k_j, v_j the stored e4m3 values, in one pass with a running m (rescaled
// only when it grows by more than 2^8).  Bound by the bytes of K and V: 2 D
// bytes and 4 D G flops a key.  64 requests of up to 8192 keys, 32 query and 8 KV
// heads of 128: 87 us, 6.05 TB/s (the plain copy reaches 6.8); 3 requests of up to
// 131072, 4 KV heads: 42 us, 5.1 TB/s, of which 12 are start-up and the spread of
// the warps' ends; 128 windows of 1024 keys, 8 KV heads of 64: 35 us, 3.8 TB/s.
//
// Split: the line of kv_sched.cuh with units of 8 or 16 rows and tiles of 32
// keys, over persistent warps.  Every KV head has the same line, so worker
// (warp) w takes head w % HKV and part w / HKV of its line: the warps of a CTA
// walk the same pages of neighbouring heads together, which reads pages stored
// token by token in rows of several heads (one head at a time, 128 B out of
// every 1 KB, ran at two thirds of that on 64 requests of up to 8192 keys).  A
// warp keeps m, l and O of its unit in registers and needs no other warp; a
// unit that one warp holds whole is written at once, parts go to the workspace,
// at most two a warp, and kv_join_kernel adds them in order (the same result
// from run to run).
//
// Products: mma.m16n8k16 on fp16, transposed: S^T = K Q^T with 16 keys by 8
// rows, O^T += V^T P^T with 16 columns by 8 rows.  tcgen05 needs 64 or 128 rows
// of A and its operands in shared memory at 16 bits; here the few rows are the
// N of the product, so none of its work is padding beyond 8 rows, and K and V
// go from their ring to registers as bytes.  e4m3 is exact in fp16; a row of Q
// is brought to fp16's upper range by a power of two (bf16 rows keep every bit
// of their leading values, what falls under fp16's 2^-24 is 2^-38 of the row's
// largest value); the K scale and the row's power go to the f32 score, the V
// scale to p before it is rounded to fp16, with a power of two that follows the
// row's largest product of the two (kv_common.cuh).
//
// Layout: no operand goes through a transpose in shared memory.  The sum over d
// may run in any order, so the thread that holds k columns 2c, 2c + 1 of key n
// takes 16 consecutive bytes of the key (one read of the swizzled tile), and Q
// is permuted to match.  Likewise the rows of O^T: thread n takes bytes
// [n D/8, (n + 1) D/8) of its four keys, and two keys' bytes are paired by one
// byte permute before the conversion.  P^T turns with one movmatrix for 8 keys.
// The ring is the warp's own: its first lane queues a tile's copies (a box a
// page) on the slot's barrier once the warp has read the slot.
#include <cuda_fp16.h>

#include "cvt.cuh"
#include "kv_cache.h"
#include "kv_common.cuh"
#include "kv_launch.h"
#include "kv_sched.cuh"
#include "sm103.cuh"

namespace ab {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
// Ring of slots (one tile each) per warp: with the 8 or 12 warps of an SM, 96 to
// 128 KB in flight; a third slot made every case 1 to 4 % slower.
constexpr int kStages = 2;
constexpr float kTop = 7.f;      // of weight_ref; with the growth below, weights stay at 2^15, in fp16
constexpr float kRescale = 8.f;  // log2 growth of a row's max, or largest weight, that triggers a rescale
// Fewest line positions of a worker: below it, more parts cost more to join
// than they save.
constexpr int kMinWork = 4;

template <int D, int NB>
struct DecCfg {
  static constexpr int RT = 8 * NB;                  // rows of a unit
  static constexpr int KT = kKvDecKeys;             // keys of a tile
  static constexpr int CTAS = D == 64 ? 3 : 2;       // resident per SM
  static constexpr int TILE = KT * D;                // bytes of K, or of V, of a tile
  static constexpr int WARP = kStages * 2 * TILE;    // a warp's ring
  static constexpr int OFF_BAR = kWarps * WARP;
  static constexpr int OFF_ABORT = OFF_BAR + kWarps * kStages * 8;
  static constexpr int SMEM = OFF_ABORT + 8;
};

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values held as one pair a lane.
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Where line position ``x`` lies: request, row tile, position in the unit.
struct Cursor {
  int n, rt, pos;
};

// All threads of a CTA: the length of the line.  A thread sums ceil(N / 128)
// consecutive requests; ``before`` (shared, kThreads entries) gets the sums
// before each thread's.
template <int RT, int KT>
__device__ __forceinline__ int64_t line_length(const KvAttnParams& p, int64_t* before) {
  __shared__ int64_t s_warp[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = (p.N + kThreads - 1) / kThreads;
  int64_t w = 0;
#pragma unroll 1  // (small code: a launch starts with a cold instruction cache)
  for (int i = 0; i < K; ++i) {
    const int64_t n = static_cast<int64_t>(tid) * K + i;
    if (n >= p.N) break;
    w += kv_request_work<RT, KT, kKvDecCost>(kv_request(static_cast<int>(n), p), p);
  }
  int64_t inc = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += a;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) base += s_warp[i];
    all += s_warp[i];
  }
  before[tid] = base + inc - w;
  __syncthreads();
  return all;
}

// A warp's cursor at position x (below the line's length).
template <int RT, int KT>
__device__ __forceinline__ Cursor locate(const KvAttnParams& p, const int64_t* before, int64_t x) {
  const int K = (p.N + kThreads - 1) / kThreads;
  int lo = 0, hi = kThreads;  // before[lo] <= x < before[lo + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= x) lo = mid;
    else hi = mid;
  }
  x -= before[lo];
  Cursor c{lo * K, 0, 0};
  KvReq r;
  while (true) {
    r = kv_request(c.n, p);
    const int64_t w = kv_request_work<RT, KT, kKvDecCost>(r, p);
    if (x < w) break;
    x -= w;
    ++c.n;
  }
  while (true) {
    const int w = kv_row_tile<RT, KT>(r, c.rt, p).n + kKvDecCost;
    if (x < w) break;
    x -= w;
    ++c.rt;
  }
  c.pos = static_cast<int>(x);
  return c;
}

template <int D, int NB, bool BF16>
__global__ void __launch_bounds__(kThreads, (DecCfg<D, NB>::CTAS))
    kv_decode_kernel(const __grid_constant__ KvMaps maps, const __grid_constant__ KvAttnParams p) {
  using C = DecCfg<D, NB>;
  constexpr int RT = C::RT, KT = C::KT;
  constexpr int NZ = KT / 16;  // 16-key groups of a tile, a page each
  constexpr int KC = D / 64;   // 16-byte chunks of a key's row per thread
  constexpr int VB = D / 8;    // bytes of a value row per thread
  constexpr int MT = D / 16;   // row tiles of O^T
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ int64_t before[kThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r8 = lane >> 2, c4 = lane & 3;
  uint8_t* const ring = sm + warp * C::WARP;
  uint64_t* const full = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR) + warp * kStages;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_ABORT);

  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kWarps * kStages; ++i) mbar_init(reinterpret_cast<uint64_t*>(sm + C::OFF_BAR) + i, 1);
    fence_mbar_init();
  }
  grid_dependency_wait();
  // The CTA's own error word: kv_join_kernel gathers them, so that no word has
  // to be cleared by a launch of its own.
  const WaitCtx wc{abort_flag, p.cta_err + blockIdx.x, p.timeout_ns};
  const bool aligned = (smem_u32(sm) & 1023u) == 0;  // the swizzled tiles need it
  const int worker = blockIdx.x * kWarps + warp, workers = gridDim.x * kWarps;
  if (tid == 0) *wc.err = aligned ? kErrNone : kErrAlign;
  if (lane == 0) p.desc[worker] = make_int4(0, 0, 0, -1);
  const int64_t total = line_length<RT, KT>(p, before);  // (its barriers publish what thread 0 wrote)
  if (!aligned || total == 0) return;
  // Parts of a head's line, at least kMinWork positions each; with more heads
  // than workers, one part and several heads a worker.
  const int64_t most = imax(1, workers / p.HKV), want = (total + kMinWork - 1) / kMinWork;
  const int parts = static_cast<int>(most < want ? most : want);
  const int g = worker / p.HKV;
  if (g >= parts) return;
  const int64_t begin = kv_part_begin(total, g, parts), end = kv_part_begin(total, g + 1, parts);
  // slots filled and read so far, as (slot, parity) of the next one
  int in_slot = 0, out_slot = 0, pending = 0;
  uint32_t out_par = 0;

  const Cursor first = locate<RT, KT>(p, before, begin);
  for (int head = worker % p.HKV; head < p.HKV; head += workers) {
  Cursor cur = first;
  KvReq rq = kv_request(cur.n, p);
  for (int64_t x = begin; x < end;) {
    // ---------------------------------------------------------- the unit and the worker's part of it
    const KvTiles kt = kv_row_tile<RT, KT>(rq, cur.rt, p);
    const int64_t unit0 = x - cur.pos;  // where the unit starts on the line
    const int64_t stop = unit0 + kKvDecCost + kt.n < end ? unit0 + kKvDecCost + kt.n : end;
    const int part0 = imax(0, cur.pos - kKvDecCost);
    const int part1 = imax(0, static_cast<int>(stop - unit0) - kKvDecCost);
    const int row0 = cur.rt * RT;
    const int rows = imin(RT, rq.R - row0);

    // Page ids of 32 16-key groups and their scales at a time: lane i holds those
    // of group i behind tile ``ld_batch`` (-1: no page, or no key that the unit sees).
    constexpr int BATCH = 32 / NZ;
    const int gb = imin(NZ, 1 << (p.page_log2 - 4));  // groups of a box of the maps
    auto key0_of = [&](int t) { return (kt.t0 + t) * KT; };
    int ld_batch = part0, ld_blk = -1;
    float ld_ks = 0.f, ld_vs = 0.f;
    auto load_ids = [&]() {
      ld_blk = -1, ld_ks = ld_vs = 0.f;
      if (ld_batch + lane / NZ < part1) {
        const int k0 = key0_of(ld_batch) + lane * 16;
        if (k0 < kt.hi && k0 + 16 > kt.lo) {
          ld_blk = p.table[cur.n * p.table_stride + (k0 >> p.page_log2)];
          if (ld_blk < 0 || ld_blk >= p.num_blocks) ld_blk = -1;
        }
      }
    };
    auto load_scales = [&]() {
      if (ld_blk >= 0) {
        const int64_t at = static_cast<int64_t>(ld_blk) * p.HKV + head;
        ld_ks = p.k_scale[at], ld_vs = p.v_scale[at];
      }
    };
    auto issue = [&](int t) {  // copies of tile t's keys into the next slot
      if (t >= part1) return;
      if (t - ld_batch == BATCH) {
        ld_batch = t;
        load_ids();
        load_scales();
      }
      // a box is a page, at most a tile: ``gb`` groups, copied where one of them has an id
      int b[NZ];
#pragma unroll
      for (int z = 0; z < NZ; ++z) b[z] = __shfl_sync(0xffffffffu, ld_blk, (t - ld_batch) * NZ + z);
      if (lane == 0) {
        int boxes = 0;
#pragma unroll
        for (int z = 0; z < NZ; ++z) {
#pragma unroll
          for (int y = 1; y < NZ - z; ++y)
            if (y < gb) b[z] = imax(b[z], b[z + y]);
          if ((z & (gb - 1)) != 0) b[z] = -1;
          boxes += b[z] >= 0 ? 1 : 0;
        }
        uint64_t* const bar = &full[in_slot];
        uint8_t* const dst = ring + in_slot * (2 * C::TILE);
        if (boxes == 0) {
          mbar_arrive(bar);
        } else {
          mbar_arrive_expect_tx(bar, boxes * gb * (2 * 16 * D));
#pragma unroll
          for (int z = 0; z < NZ; ++z)
            if (b[z] >= 0) {
              const int s0 = (key0_of(t) + 16 * z) & ((1 << p.page_log2) - 1);
              tma_load_4d(dst + z * 16 * D, &maps.k, bar, 0, head, s0, b[z]);
              tma_load_4d(dst + C::TILE + z * 16 * D, &maps.v, bar, 0, head, s0, b[z]);
            }
        }
      }
      in_slot = in_slot + 1 == kStages ? 0 : in_slot + 1;
      ++pending;
    };
    load_ids();
#pragma unroll
    for (int i = 0; i < kStages; ++i) issue(part0 + i);
    load_scales();

    // Q in fp16: the thread holds row r8 of each 8 rows; the scores of a thread
    // belong to rows 2 c4 and 2 c4 + 1
    int lo[NB][2], hi[NB][2];
    float rs[NB][2];
    uint32_t qb[NB][KC * 4][2];  // [8 rows][k step][b0, b1]
#pragma unroll
    for (int e = 0; e < NB; ++e) {
      const int r = r8 + 8 * e;
      const bool live = r < rows;
      const int i = (row0 + r) / p.G, gq = (row0 + r) % p.G;
      const uint8_t* src = p.q + 2 * ((static_cast<int64_t>(rq.a) + i) * p.sq_s +
                                      static_cast<int64_t>(head * p.G + gq) * p.sq_h);
      uint32_t w[KC][8];
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint4 x4 = make_uint4(0u, 0u, 0u, 0u);
          if (live) x4 = *reinterpret_cast<const uint4*>(src + 2 * ((c4 * KC + c) * 16 + u * 8));
          w[c][4 * u] = x4.x, w[c][4 * u + 1] = x4.y, w[c][4 * u + 2] = x4.z, w[c][4 * u + 3] = x4.w;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float2 f = unpack2<BF16>(w[c][u]);
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float back;
      const float up = to_top(amax, &back);
      back *= p.scale_log2;
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float2 f = unpack2<BF16>(w[c][u]);
          // bytes 4j .. 4j + 3 of the chunk are k step 4c + j: pairs (0,1) and (2,3)
          qb[e][c * 4 + u / 2][u & 1] = pack2<false>(f.x * up, f.y * up);
        }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int rr = 8 * e + 2 * c4 + y;
        rs[e][y] = __shfl_sync(0xffffffffu, back, (2 * c4 + y) * 4);
        lo[e][y] = hi[e][y] = 0;
        if (rr < rows) kv_row_keys(rq, (row0 + rr) / p.G, p.causal, p.window, &lo[e][y], &hi[e][y]);
      }
    }
    // keys that every live row sees lie in [lo_all, hi_all)
    int lo_all, hi_all, xx;
    kv_row_keys(rq, (row0 + rows - 1) / p.G, p.causal, p.window, &lo_all, &xx);
    kv_row_keys(rq, row0 / p.G, p.causal, p.window, &xx, &hi_all);

    // A row's scores are kept relative to nm (its m, 0 before its first key)
    // and compared with th (kRescale, -inf before its first key); its weights and
    // O are at 2^ref.
    float nm[NB][2], th[NB][2], l[NB][2], ref[NB][2];
    float o[NB][MT][4];
#pragma unroll
    for (int e = 0; e < NB; ++e) {
      nm[e][0] = nm[e][1] = l[e][0] = l[e][1] = 0.f;
      th[e][0] = th[e][1] = -INFINITY;
      ref[e][0] = ref[e][1] = kKvRefNone;
#pragma unroll
      for (int t = 0; t < MT; ++t) o[e][t][0] = o[e][t][1] = o[e][t][2] = o[e][t][3] = 0.f;
    }

    float ks_l = 0.f, lv_l = 0.f;  // K scales, log2 of the V scales of the 32 groups
    int cp_blk = -1;               // being computed, and their ids
    int cp_batch = part0 - BATCH;
    bool ok = true;
    for (int t = part0; t < part1; ++t) {
      if (t - cp_batch == BATCH) {  // (the copies are kStages tiles ahead: in this batch already)
        cp_batch = t;
        cp_blk = ld_blk, ks_l = ld_ks, lv_l = log2f(ld_vs);
      }
      float ks[NZ], lv[NZ];
      bool have[NZ], any = false, edge = false;
#pragma unroll
      for (int z = 0; z < NZ; ++z) {
        const int from = (t - cp_batch) * NZ + z;
        ks[z] = __shfl_sync(0xffffffffu, ks_l, from), lv[z] = __shfl_sync(0xffffffffu, lv_l, from);
        have[z] = __shfl_sync(0xffffffffu, cp_blk, from) >= 0;
        any |= have[z], edge |= !have[z];
      }
      if (!(ok = mbar_wait_warp(&full[out_slot], out_par, wc, kErrWaitKV))) break;
      const uint8_t* const st = ring + out_slot * (2 * C::TILE);
      if (++out_slot == kStages) out_slot = 0, out_par ^= 1;
      --pending;
      if (any) {
        const int k0 = key0_of(t);
        edge |= k0 < lo_all || k0 + KT > hi_all;
        // ---- S^T of 16 keys by 8 NB rows, in two chains
        float s[NZ][NB][4];
#pragma unroll
        for (int z = 0; z < NZ; ++z) {
          float s2[NB][2][4];
#pragma unroll
          for (int e = 0; e < NB; ++e)
#pragma unroll
            for (int y = 0; y < 2; ++y) s2[e][y][0] = s2[e][y][1] = s2[e][y][2] = s2[e][y][3] = 0.f;
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const uint4 x0 = *reinterpret_cast<const uint4*>(st + kv_chunk_at<D>(16 * z + r8, c4 * KC + c));
            const uint4 x8 = *reinterpret_cast<const uint4*>(st + kv_chunk_at<D>(16 * z + r8 + 8, c4 * KC + c));
            const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w8[4] = {x8.x, x8.y, x8.z, x8.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t a[4];
              e4m3x4_to_f16(w0[u], &a[0], &a[2]);
              e4m3x4_to_f16(w8[u], &a[1], &a[3]);
#pragma unroll
              for (int e = 0; e < NB; ++e) mma16816(s2[e][u & 1], a, qb[e][c * 4 + u][0], qb[e][c * 4 + u][1]);
            }
          }
#pragma unroll
          for (int e = 0; e < NB; ++e)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              s[z][e][y] = (s2[e][0][y] + s2[e][1][y]) * (ks[z] * rs[e][y & 1]) - nm[e][y & 1];
        }
        if (edge) {
#pragma unroll
          for (int z = 0; z < NZ; ++z)
#pragma unroll
            for (int e = 0; e < NB; ++e)
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int k = k0 + 16 * z + r8 + 8 * (y >> 1);
                if (!have[z] || k < lo[e][y & 1] || k >= hi[e][y & 1]) s[z][e][y] = -INFINITY;
              }
        }
        // ---- a max or a weight that grew past its threshold: rescale the row
        auto most = [&](int z, int e, int y) {  // score, relative to nm, up to which neither did
          return fminf(th[e][y], kTop + kRescale - (lv[z] + ref[e][y]));
        };
        bool grew = false;
#pragma unroll
        for (int z = 0; z < NZ; ++z)
#pragma unroll
          for (int e = 0; e < NB; ++e) {
            const float m0 = most(z, e, 0), m1 = most(z, e, 1);
            grew |= s[z][e][0] > m0 || s[z][e][1] > m1 || s[z][e][2] > m0 || s[z][e][3] > m1;
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int e = 0; e < NB; ++e) {
            float f[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              // the row's largest score, weight (log2) and excess over a threshold
              float mx = -INFINITY, top = -INFINITY, over = -INFINITY;
#pragma unroll
              for (int z = 0; z < NZ; ++z) {
                const float x = fmaxf(s[z][e][y], s[z][e][2 + y]);
                mx = fmaxf(mx, x), top = fmaxf(top, x + lv[z]), over = fmaxf(over, x - most(z, e, y));
              }
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                over = fmaxf(over, __shfl_xor_sync(0xffffffffu, over, d));
              }
              f[y] = 1.f;
              if (over > 0.f) {  // (row by row, so that no row's result depends on another's)
                const bool first = th[e][y] == -INFINITY;
                const float up = mx > th[e][y] ? mx : 0.f;
                // the largest weight: this tile's or, as it was where ref was set, an earlier one's
                const float now = weight_ref(kTop, first ? top - up : fmaxf(top, kTop - ref[e][y]) - up);
                f[y] = first ? 0.f : ex2(now - ref[e][y] - up);
                l[e][y] *= first ? 0.f : ex2(-up);
                ref[e][y] = now;
                nm[e][y] += up;
                th[e][y] = kRescale;
#pragma unroll
                for (int z = 0; z < NZ; ++z) s[z][e][y] -= up, s[z][e][2 + y] -= up;
              }
            }
#pragma unroll
            for (int u = 0; u < MT; ++u)
              o[e][u][0] *= f[0], o[e][u][1] *= f[1], o[e][u][2] *= f[0], o[e][u][3] *= f[1];
          }
        }
        uint32_t pb[NZ][NB][2];
#pragma unroll
        for (int z = 0; z < NZ; ++z) {
#pragma unroll
          for (int e = 0; e < NB; ++e) {
            const float w0 = weight_factor(lv[z], ref[e][0]), w1 = weight_factor(lv[z], ref[e][1]);
            const float p0 = ex2(s[z][e][0]), p1 = ex2(s[z][e][1]), p2 = ex2(s[z][e][2]), p3 = ex2(s[z][e][3]);
            l[e][0] += p0 + p2;
            l[e][1] += p1 + p3;
            pb[z][e][0] = turn8x8(pack2<false>(p0 * w0, p1 * w1));
            pb[z][e][1] = turn8x8(pack2<false>(p2 * w0, p3 * w1));
          }
        }
        // ---- O^T += V^T P^T
        constexpr int VW = VB / 4;
#pragma unroll
        for (int z = 0; z < NZ; ++z) {
          uint32_t vw[4][VW];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = 16 * z + 2 * c4 + (e & 1) + 8 * (e >> 1);
            const uint8_t* const at = st + C::TILE + kv_chunk_at<D>(key, r8 * VB / 16) + (r8 * VB) % 16;
            if constexpr (VB == 16) {
              const uint4 w = *reinterpret_cast<const uint4*>(at);
              vw[e][0] = w.x, vw[e][1] = w.y, vw[e][2] = w.z, vw[e][3] = w.w;
            } else {
              const uint2 w = *reinterpret_cast<const uint2*>(at);
              vw[e][0] = w.x, vw[e][1] = w.y;
            }
          }
          if (edge) {  // a zero P times a NaN byte would be NaN: keys that no row sees are zeroed
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = k0 + 16 * z + 2 * c4 + (e & 1) + 8 * (e >> 1);
              if (!have[z] || k < kt.lo || k >= kt.hi) {
#pragma unroll
                for (int u = 0; u < VW; ++u) vw[e][u] = 0u;
              }
            }
          }
#pragma unroll
          for (int u = 0; u < VW; ++u) {
            // bytes 4u .. 4u + 3 of keys (0, 1) and (2, 3) paired; byte 2i is row r8 of tile i, 2i + 1 its row r8 + 8
            uint32_t a[2][4];
            e4m3x4_to_f16(__byte_perm(vw[0][u], vw[1][u], 0x5140), &a[0][0], &a[0][1]);
            e4m3x4_to_f16(__byte_perm(vw[0][u], vw[1][u], 0x7362), &a[1][0], &a[1][1]);
            e4m3x4_to_f16(__byte_perm(vw[2][u], vw[3][u], 0x5140), &a[0][2], &a[0][3]);
            e4m3x4_to_f16(__byte_perm(vw[2][u], vw[3][u], 0x7362), &a[1][2], &a[1][3]);
#pragma unroll
            for (int e = 0; e < NB; ++e)
#pragma unroll
              for (int y = 0; y < 2; ++y) mma16816(o[e][2 * u + y], a[y], pb[z][e][0], pb[z][e][1]);
          }
        }
      }
      __syncwarp();            // every lane has read the slot,
      issue(t + kStages);      // which is filled again
    }

    if (!ok) {  // a wait that ran out: the copies in flight land before the warp leaves
      if (lane == 0)
        for (int i = 0; i < pending; ++i)
          mbar_drain(&full[(out_slot + i) % kStages], out_par ^ (out_slot + i >= kStages ? 1u : 0u));
      return;
    }

    // ---------------------------------------------------------- the unit's rows, or my part of them
    if (part1 > part0) {
      const bool whole = part0 == 0 && part1 == kt.n;
      const int slot = 2 * worker + (part0 > 0 ? 0 : 1);
#pragma unroll
      for (int e = 0; e < NB; ++e)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float sum = l[e][y];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          const int row = 8 * e + 2 * c4 + y;
          if (row >= rows) continue;
          // columns [r8 VB, (r8 + 1) VB)
          const float back = ex2(-ref[e][y]);
          const float f = whole ? (sum == 0.f ? 0.f : back / sum) : back;
          float v[VB];
#pragma unroll
          for (int u = 0; u < MT; ++u) v[2 * u] = o[e][u][y] * f, v[2 * u + 1] = o[e][u][2 + y] * f;
          if (whole) {
            const int64_t at = static_cast<int64_t>(rq.a) + (row0 + row) / p.G;
            const int hq = head * p.G + (row0 + row) % p.G;
            store_o<BF16, VB>(p, at, hq, r8 * VB, v);
            if (r8 == 0) store_lse(p, at, hq, nm[e][y], sum);
          } else {
            float* const to = p.part_o + (static_cast<int64_t>(slot) * RT + row) * D + r8 * VB;
#pragma unroll
            for (int u = 0; u < VB; u += 4)
              *reinterpret_cast<float4*>(to + u) = make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
            if (r8 == 0) p.part_ml[slot * RT + row] = make_float2(nm[e][y], sum);
          }
        }
      if (lane == 0 && part0 > 0 && part1 == kt.n) {  // ends a unit that part g0 began
        const int g0 = kv_part_of(total, unit0 + kKvDecCost, parts);
        p.desc[worker] = make_int4(rq.a, row0, head << 16 | rows, g0);
      }
    }

    // ---------------------------------------------------------- next unit
    x = stop;
    cur.pos = 0;
    if (x < end && ++cur.rt == kv_row_tiles<RT>(rq)) {
      cur.rt = 0;
      do {
        rq = kv_request(++cur.n, p);
      } while (rq.R == 0);
    }
  }
  }
}

template <int D, int NB, bool BF16>
cudaError_t launch_nb(const KvAttnParams& p, const KvMaps& maps, int sms, KvJoinPart* left, cudaStream_t st) {
  using C = DecCfg<D, NB>;
  auto kern = kv_decode_kernel<D, NB, BF16>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem_once(kern, C::SMEM, &done);
  if (e != cudaSuccess) return e;
  const int grid = imin(sms * C::CTAS, kKvDecMaxRows / (2 * kWarps * C::RT));
  *left = kv_join_part(p, grid * kWarps, grid, p.HKV, C::RT);
  return launch_chained(kern, grid, kThreads, C::SMEM, st, maps, p);
}

// Units of 8 rows where a request's rows (by the mean number of its queries)
// fit them, of 16 otherwise; either serves any number.
template <int D, bool BF16>
cudaError_t launch_t(const KvAttnParams& p, const KvMaps& maps, int sms, KvJoinPart* left, cudaStream_t st) {
  const int64_t mean = (static_cast<int64_t>(p.T) + p.N - 1) / p.N;
  return mean * p.G <= 8 ? launch_nb<D, 1, BF16>(p, maps, sms, left, st) : launch_nb<D, 2, BF16>(p, maps, sms, left, st);
}

}  // namespace

cudaError_t launch_kv_decode(const KvAttnParams& p, const KvMaps& maps, bool bf16, int sms, KvJoinPart* left,
                             cudaStream_t st) {
  if (p.D == 64) return bf16 ? launch_t<64, true>(p, maps, sms, left, st) : launch_t<64, false>(p, maps, sms, left, st);
  return bf16 ? launch_t<128, true>(p, maps, sms, left, st) : launch_t<128, false>(p, maps, sms, left, st);
}

}  // namespace ab
