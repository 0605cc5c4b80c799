// Attention over the paged 8-bit cache for many rows (query, head of the group)
// per KV head: prompts and chunks of prompts against what is cached of them.
//
// The mathematics of kv_decode.cu, on tcgen05 as in the dense forward: units of
// two 128-row tiles of one KV head, key blocks of 128,
//   S_w = Q_w K_j^T in tensor memory, P_w = 2^(S_w f - m) back into it as the
//   fp16 A operand of O_w += P_w V_j,
// two softmax warpgroups, one row a thread, O rescaled only when P outgrows
// fp16.  P goes to the products in halves of 64 keys, so that P V of the first
// runs while the softmax works on the second.  Rows are packed (query, head), so a group's heads
// share each key block and short chunks fill the tiles.
//
// Bound by the tensor cores and the exponentials, with the bytes of K and V a
// small part; what is new against the dense forward is that the operands have
// to be made.  2048 + 1713 tokens on 14336 cached ones, 32 query and 8 KV heads of
// 128: 514 us, 1.20 PFLOP/s, 62 % of the measured peak, held back by the issue of
// the products (below).  TMA brings pages as bytes into a raw ring; four warps convert them
// to fp16 (exact) in the 128-byte-swizzled tiles that the products read.  A
// block's page scales (at most one per 16 keys) are applied by the softmax, 16
// columns at a time: K's as factors of the f32 scores, V's in the exponent, so that
// the power is the weight P vs 2^ref (kv_common.cuh) that is rounded to fp16; its
// sum over 16 columns, divided by vs, goes into l, which is kept at 2^ref as well.
// (A product of P with the scale for each weight took 3 % longer.)  Each
// softmax thread loads its own row of Q, brings it to fp16's upper range by a
// power of two and writes it into the swizzled Q tile.
//
// Work: the line of kv_sched.cuh over all heads, cut evenly over one CTA per
// SM; at most two parts of units per CTA go through the workspace.
//
// Warp roles (16 warps): 0-3 softmax of tile 0, 4-7 of tile 1, 8 copies, 9 MMA
// issue, 10 the walk along the line, a unit ahead of the others (it publishes
// units through a two-slot ring), 11 idle, 12-13
// conversion of K, 14-15 of V.  Every wait is bounded.
#include <cuda_fp16.h>

#define AB_INLINE_WAITS 1
#include "cvt.cuh"
#include "kv_cache.h"
#include "kv_common.cuh"
#include "kv_launch.h"
#include "kv_sched.cuh"
#include "sm103.cuh"

namespace ab {

namespace {

constexpr int BQ = 128, RT = kKvPrRows, KT = kKvPrKeys, COST = kKvPrCost;
constexpr int kWarps = 16, THREADS = kWarps * 32;
// launched at 128 registers a thread, re-split per warpgroup: the softmax
// warpgroups hold 64 scores and 32 P pairs a thread
constexpr uint32_t REG_SOFT = 168, REG_CTL = 88, REG_CONV = 88;
static_assert(2 * REG_SOFT + REG_CTL + REG_CONV == 4 * 128, "register split must equal the launch's registers");
constexpr float kMostSum = 32768.f;  // of half a block's P, or weights, before a row's max is taken anew
// Of weight_ref.  The room from here to kMostSum decides how often a row's max is taken
// anew: the chunk case takes 528 us at 0 to 3, 531 to 536 at 4, 548 at 6, 556 at 7, cross
// attention 57.7, 58.5, 59.2, 62.8, 63.7.
constexpr float kTop = 3.f;
// Largest |log2| of a V scale whose weights' sum gives l: the weights of P down to
// 2^-36 then stay above f32's 2^-126 while ref is -45 or more.  A group with another
// (0, or 2^-100 of a page of zeros), or a row with a smaller ref, sends its half
// block through the slow path.
constexpr float kFarScale = 45.f;
// Largest sum of a half block's P at 2^ref that goes into l as it is (l, a sum of one
// for each 64 keys, stays finite at any ref); -1: none does.
__device__ __forceinline__ float most_sum(float ref) {
  return ref < -kFarScale ? -1.f : fminf(kMostSum * ex2(ref), 0x1p109f);
}
constexpr int kGroups = KT / 16;  // 16-key groups of a block: a page scale each
constexpr int HK = 64;            // keys of a half block
static_assert(KT == 2 * HK && kGroups == 8, "a half block's scales are one 16-byte load");
constexpr int kScaleRing = 16;    // blocks of scales; the copies run at most 8 ahead of the softmax

// mma_ss_w and mma_ts_w with the lane elected beforehand (``elected``: elect_lane(),
// not 0 in one lane): an issuing warp that shares its scheduler with busy warps is slowed
// by every instruction.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t x;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(x));
  return x;
}
__device__ __forceinline__ void mma_ss_e(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(elected));
}
__device__ __forceinline__ void mma_ts_e(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(elected));
}

template <int D>
struct PrCfg {
  static constexpr int NSLAB = D / 64;
  static constexpr int QSLAB = 128 * 128;        // [128 rows x 64 columns] fp16, 128-byte swizzled
  static constexpr int QTILE = NSLAB * QSLAB;    // a tile of Q
  static constexpr int SLAB = KT * 128;          // [128 keys x 64 columns]
  static constexpr int TILE = NSLAB * SLAB;      // a block's K or V
  static constexpr int RAW = KT * D;             // the same as bytes
  static constexpr int NT = D == 64 ? 6 : 3;     // ring of converted tiles, K and V in turn
  static constexpr int NR = D == 64 ? 8 : 4;     // ring of raw tiles, K and V in turn
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_T = OFF_Q + 2 * QTILE;
  static constexpr int OFF_RAW = OFF_T + NT * TILE;
  static constexpr int OFF_UNIT = OFF_RAW + NR * RAW;   // 2 unit descriptors of 64 bytes
  static constexpr int OFF_SC = OFF_UNIT + 2 * 64;      // K scales, log2 of V scales and their inverses, [kScaleRing][kGroups] each
  static constexpr int OFF_BAR = OFF_SC + 3 * kScaleRing * kGroups * 4;
  static constexpr int OFF_MISC = OFF_BAR + 56 * 8;
  static constexpr int OFF_WORK = OFF_MISC + 32;        // the line's length, a share of the requests per warp
  static constexpr int SMEM = OFF_WORK + kWarps * 8;    // (all of it: nothing static beside the 1024-byte aligned tiles)
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
  static constexpr uint32_t T_S = 0, T_O = 256;  // tile w: scores at 128 w, O at 256 + D w
};

enum PrBar : int {
  Q_FULL0 = 0,                 // per tile: 4 softmax warps wrote Q
  RAW_FULL0 = Q_FULL0 + 2,     // NR
  RAW_EMPTY0 = RAW_FULL0 + 8,  // NR: 2 conversion warps read it
  T_FULL0 = RAW_EMPTY0 + 8,    // NT: 2 conversion warps wrote it
  T_EMPTY0 = T_FULL0 + 6,      // NT: its products have completed
  S_FULL0 = T_EMPTY0 + 6,      // per tile
  P_READY0 = S_FULL0 + 2,      // per tile and half: 4 softmax warps stored P
  O_DONE0 = P_READY0 + 4,      // per tile and half: its P V, and all before it, completed
  O_FREE0 = O_DONE0 + 4,       // per tile: 4 softmax warps read the unit's O rows
  UNIT_FULL0 = O_FREE0 + 2,    // 2 slots
  UNIT_EMPTY0 = UNIT_FULL0 + 2,  // 2 slots: the 14 other working warps read it
  DRAIN = UNIT_EMPTY0 + 2,
  NUM_BARS
};
static_assert(NUM_BARS <= 56, "barrier storage");

// A unit, or the CTA's part of one: key blocks [j0, j1).
struct PrUnit {
  int n, a, nq, L, off, R;  // the request (kv_sched.cuh)
  int row0, head;
  int j0, j1;            // j0 == j1: no block, its rows are zero
  int lo, hi;            // keys that some row of the unit sees
  int slot;              // -1: the whole unit, else the slot of its partial rows
  int valid;
};
static_assert(sizeof(PrUnit) <= 64, "descriptor slot");

// Key blocks [lo, hi) of tile w of the unit, within its part, and the keys that
// all its live rows see.
struct PrTile {
  int lo, hi, all_lo, all_hi;
};

__device__ __forceinline__ PrTile tile_of(const PrUnit& u, int w, const KvAttnParams& p) {
  PrTile t{0, 0, 0, 0};
  const int r0 = u.row0 + w * BQ, r1 = imin(u.R, r0 + BQ);
  if (r0 >= r1) return t;
  KvReq r{u.a, u.nq, u.L, u.off, u.R};
  int lo, hi;
  kv_row_keys(r, r0 / p.G, p.causal, p.window, &lo, &t.all_hi);
  kv_row_keys(r, (r1 - 1) / p.G, p.causal, p.window, &t.all_lo, &hi);
  if (hi <= lo) return t;
  t.lo = imax(lo / KT, u.j0), t.hi = imin((hi + KT - 1) / KT, u.j1);
  if (t.hi < t.lo) t.lo = t.hi = 0;
  return t;
}

// ---------------------------------------------------------------- the walk
// (one warp; every lane holds the same cursor)

struct PrCursor {
  int n, rt, head, pos;
};

// Positions of a request on the line of one head, all lanes together.
__device__ __forceinline__ int64_t lanes_work(const KvAttnParams& p, const KvReq& r) {
  int64_t w = 0;
  const int nt = kv_row_tiles<RT>(r);
  for (int rt = threadIdx.x & 31; rt < nt; rt += 32) w += kv_row_tile<RT, KT>(r, rt, p).n + COST;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  return w;
}

template <typename T>
__device__ __forceinline__ T warp_uniform(T x) {
  return __shfl_sync(0xffffffffu, x, 0);
}

// Calls f(n, request) for the requests of [n0, n1) that have rows here, in
// order, until it returns true; 32 requests are looked up at once.
template <typename F>
__device__ __forceinline__ void each_request(const KvAttnParams& p, int n0, int n1, F f) {
  const int lane = threadIdx.x & 31;
  for (int b = n0; b < n1; b += 32) {
    KvReq mine{};
    if (b + lane < n1) mine = kv_request(b + lane, p);
    for (uint32_t m = __ballot_sync(0xffffffffu, mine.R > 0); m != 0; m &= m - 1) {
      const int src = __ffs(m) - 1;
      KvReq r;
      r.a = __shfl_sync(0xffffffffu, mine.a, src), r.nq = __shfl_sync(0xffffffffu, mine.nq, src);
      r.L = __shfl_sync(0xffffffffu, mine.L, src), r.off = __shfl_sync(0xffffffffu, mine.off, src);
      r.R = __shfl_sync(0xffffffffu, mine.R, src);
      if (f(b + src, r)) return;
    }
  }
}

// Cursor of position x counted from request n0 (all heads).
__device__ __forceinline__ PrCursor walk_to(const KvAttnParams& p, int n0, int64_t x) {
  const int lane = threadIdx.x & 31;
  PrCursor c{n0, 0, 0, 0};
  each_request(p, n0, p.N, [&](int n, const KvReq& r) {
    c.n = n;
    const int64_t w = lanes_work(p, r) * p.HKV;
    if (x < w) return true;
    x -= w;
    return false;
  });
  const KvReq r = kv_request(c.n, p);
  const int nt = kv_row_tiles<RT>(r);
  for (int b = 0;; b += 32) {
    const int n = b + lane < nt ? kv_row_tile<RT, KT>(r, b + lane, p).n + COST : 0;
    const int64_t w = static_cast<int64_t>(n) * p.HKV;
    int64_t inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, x < inc);
    if (past == 0) {
      x -= __shfl_sync(0xffffffffu, inc, 31);
      continue;
    }
    const int src = __ffs(past) - 1;
    x -= __shfl_sync(0xffffffffu, inc - w, src);
    const int size = __shfl_sync(0xffffffffu, n, src);
    c.rt = b + src;
    c.head = static_cast<int>(x / size);
    c.pos = static_cast<int>(x % size);
    return c;
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS, 1) kv_prompt_kernel(const __grid_constant__ KvMaps maps,
                                                               const __grid_constant__ KvAttnParams p) {
  using C = PrCfg<D>;
  extern __shared__ __align__(1024) uint8_t sm[];
  int64_t* const s_work = reinterpret_cast<int64_t*>(sm + C::OFF_WORK);
  uint64_t* const bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 8);
  PrUnit* const units = reinterpret_cast<PrUnit*>(sm + C::OFF_UNIT);
  float* const k_scales = reinterpret_cast<float*>(sm + C::OFF_SC);               // [kScaleRing][kGroups]; -1: no page
  float* const v_logs = k_scales + kScaleRing * kGroups;
  float* const v_invs = v_logs + kScaleRing * kGroups;  // NaN: far (kFarScale)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  grid_dependency_wait();
  const WaitCtx wc{abort_flag, p.cta_err + blockIdx.x, p.timeout_ns};
  // a unit lasts as long as its keys do: waits for one to begin or to be taken
  // have a limit of their own (any wait that runs out ends the others too)
  const WaitCtx wu{abort_flag, p.cta_err + blockIdx.x, 64 * p.timeout_ns};
  const bool aligned = (smem_u32(sm) & 1023u) == 0;
  if (threadIdx.x == 0) {
    *wc.err = aligned ? kErrNone : kErrAlign;
    p.desc[blockIdx.x] = make_int4(0, 0, 0, -1);
    *abort_flag = 0;
  }
  // ---------------------------------------------------------------- the line, and the CTA's part of it
  const int per = (p.N + kWarps - 1) / kWarps;
  {
    int64_t w = 0;
    each_request(p, imin(p.N, warp * per), imin(p.N, (warp + 1) * per), [&](int, const KvReq& r) {
      w += lanes_work(p, r) * p.HKV;
      return false;
    });
    if (lane == 0) s_work[warp] = w;
  }
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) total += s_work[i];
  if (!aligned || total == 0) return;
  const int64_t want = (total + kKvPrMinWork - 1) / kKvPrMinWork;
  const int parts = want < static_cast<int64_t>(gridDim.x) ? static_cast<int>(want) : static_cast<int>(gridDim.x);
  if (static_cast<int>(blockIdx.x) >= parts) return;
  const int64_t begin = kv_part_begin(total, blockIdx.x, parts), end = kv_part_begin(total, blockIdx.x + 1, parts);

  // ---------------------------------------------------------------- set-up
  if (threadIdx.x == 0) {
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bars[Q_FULL0 + w], 4);
      mbar_init(&bars[S_FULL0 + w], 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars[P_READY0 + 2 * w + b], 4);
        mbar_init(&bars[O_DONE0 + 2 * w + b], 1);
      }
      mbar_init(&bars[O_FREE0 + w], 4);
      mbar_init(&bars[UNIT_FULL0 + w], 1);
      mbar_init(&bars[UNIT_EMPTY0 + w], 14);
    }
    for (int i = 0; i < C::NR; ++i) {
      mbar_init(&bars[RAW_FULL0 + i], 1);
      mbar_init(&bars[RAW_EMPTY0 + i], 2);
    }
    for (int i = 0; i < C::NT; ++i) {
      mbar_init(&bars[T_FULL0 + i], 2);
      mbar_init(&bars[T_EMPTY0 + i], 1);
    }
    mbar_init(&bars[DRAIN], 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto finish = [&]() {
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
    if (warp == 9) {
      __syncwarp();
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
  };
  // the uc-th unit of this CTA
  auto next_unit = [&](uint32_t uc, bool* okp) -> PrUnit {
    const uint32_t slot = uc & 1;
    PrUnit u{};
    if (!(*okp = mbar_wait_warp(&bars[UNIT_FULL0 + slot], (uc >> 1) & 1, wu, kErrWaitTile))) return u;
    u = units[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[UNIT_EMPTY0 + slot]);
    return u;
  };

  if (warp >= 12) {
    // ============================================================ conversion: two warps for K, two for V
    // A lane takes 16 bytes of a row (16 values) and writes two 16-byte chunks of
    // fp16.  Eight lanes (one shared-memory phase) hold rows r and r ^ 5 of an
    // 8-row group: reads then fall in different halves of the 128-byte lines and
    // writes on chunks of different parity, without bank conflicts.
    setmaxnreg_dec<REG_CONV>();
    const int kv = (warp - 12) >> 1, cw = (warp - 12) & 1;
    const int row8 = (lane >> 3) ^ (((lane >> 2) & 1) * 5), c4 = lane & 3;
    uint32_t bc = 0;
    bool ok = true;
    for (uint32_t uc = 0; ok; ++uc) {
      const PrUnit u = next_unit(uc, &ok);
      if (!ok || !u.valid) break;
      if (u.valid == 2) continue;
      for (int j = u.j0; j < u.j1; ++j, ++bc) {
        const uint32_t ic = 2 * bc + kv;
        const int rs = ic % C::NR, ts = ic % C::NT;
        const uint32_t n = ic / C::NT;
        if (!(ok = mbar_wait_warp(&bars[RAW_FULL0 + rs], (ic / C::NR) & 1, wc, kErrWaitStage))) break;
        if (n >= 1 && !(ok = mbar_wait_warp(&bars[T_EMPTY0 + ts], (n - 1) & 1, wc, kErrWaitKVFree))) break;
        const uint8_t* const raw = sm + C::OFF_RAW + rs * C::RAW;
        uint8_t* const out = sm + C::OFF_T + ts * C::TILE;
        // V rows that no query sees are zeroed: a zero P times a NaN would be NaN
        bool edge = false;
        if (kv) {
          edge = j * KT < u.lo || (j + 1) * KT > u.hi;
          const float* const ksc = k_scales + (bc % kScaleRing) * kGroups;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) edge |= ksc[g] < 0.f;
        }
#pragma unroll 2
        for (int it = 0; it < KT / 16; ++it) {  // 8 rows
          const int row = cw * (KT / 2) + it * 8 + row8;
          uint4 x[C::NSLAB];
#pragma unroll
          for (int s = 0; s < C::NSLAB; ++s)
            x[s] = *reinterpret_cast<const uint4*>(raw + kv_chunk_at<D>(row, s * 4 + c4));
          if (edge) {
            const int key = j * KT + row;
            const bool page = k_scales[(bc % kScaleRing) * kGroups + (row >> 4)] >= 0.f;
            if (!page || key < u.lo || key >= u.hi) {
#pragma unroll
              for (int s = 0; s < C::NSLAB; ++s) x[s] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
#pragma unroll
          for (int s = 0; s < C::NSLAB; ++s) {
            const uint32_t xs[4] = {x[s].x, x[s].y, x[s].z, x[s].w};
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_to_f16(xs[e], &y[2 * e], &y[2 * e + 1]);
            uint8_t* const slab = out + s * C::SLAB;
            *reinterpret_cast<uint4*>(slab + sw128_offset(row, 2 * c4)) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(slab + sw128_offset(row, 2 * c4 + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[RAW_EMPTY0 + rs]);
          mbar_arrive(&bars[T_FULL0 + ts]);
        }
      }
    }
    finish();
    return;
  }
  if (warp >= 8) {
    setmaxnreg_dec<REG_CTL>();
    if (warp == 10) {
      // ============================================================ the walk
      int w0 = 0;
      int64_t x = begin;
      while (x >= s_work[w0]) x -= s_work[w0++];
      PrCursor cur = walk_to(p, w0 * per, x);
      KvReq rq = kv_request(cur.n, p);
      x = begin;
      for (uint32_t uc = 0;; ++uc) {
        PrUnit u{};
        int64_t stop = x;
        u.valid = x < end;
        if (u.valid) {
          const KvTiles kt = kv_row_tile<RT, KT>(rq, cur.rt, p);
          const int64_t unit0 = x - cur.pos;
          stop = unit0 + COST + kt.n < end ? unit0 + COST + kt.n : end;
          const int part0 = imax(0, cur.pos - COST), part1 = imax(0, static_cast<int>(stop - unit0) - COST);
          const bool whole = part0 == 0 && part1 == kt.n;
          u.n = cur.n, u.a = rq.a, u.nq = rq.nq, u.L = rq.L, u.off = rq.off, u.R = rq.R;
          u.row0 = cur.rt * RT, u.head = cur.head;
          u.lo = kt.lo, u.hi = kt.hi;
          u.j0 = kt.t0 + part0;
          u.j1 = kt.hi > kt.lo ? kt.t0 + part1 : u.j0;  // (a unit that sees nothing has no block)
          u.slot = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (part0 > 0 ? 0 : 1);
          if (part1 <= part0) u.valid = 2;  // only start-up positions: nothing to do
          if (lane == 0 && part0 > 0 && part1 == kt.n) {
            const int g0 = kv_part_of(total, unit0 + COST, parts);
            p.desc[blockIdx.x] = make_int4(rq.a, u.row0, cur.head << 16 | imin(RT, rq.R - u.row0), g0);
          }
        }
        const uint32_t slot = uc & 1;
        if (uc >= 2 && !mbar_wait_warp(&bars[UNIT_EMPTY0 + slot], ((uc >> 1) - 1) & 1, wu, kErrWaitTile)) break;
        if (lane == 0) {
          units[slot] = u;
          mbar_arrive(&bars[UNIT_FULL0 + slot]);
        }
        if (!u.valid) break;
        x = stop;
        cur.pos = 0;
        if (x < end && ++cur.head == p.HKV) {
          cur.head = 0;
          if (++cur.rt == kv_row_tiles<RT>(rq)) {
            cur.rt = 0;
            do {
              rq = kv_request(++cur.n, p);
            } while (rq.R == 0);
          }
        }
      }
    } else if (warp == 8) {
      // ============================================================ copies
      // Lane i looks up 16-key group i of four blocks (page ids and scales four
      // blocks ahead); the first lane of a page that has seen keys copies it.
      const int gp = 1 << (p.page_log2 - 4);  // groups a page
      const uint32_t page_lanes = ((1u << gp) - 1u) << (lane & ~(gp - 1));
      uint32_t ic = 0;  // raw tiles so far
      bool ok = true;
      for (uint32_t uc = 0; ok; ++uc) {
        const PrUnit u = next_unit(uc, &ok);
        if (!ok || !u.valid) break;
        if (u.valid == 2) continue;
        const int k_end = imin(u.hi, u.j1 * KT);
        auto look_up = [&](int k0) {  // table entry of keys [k0, k0 + 16), -1 where nothing is seen
          return k0 >= k_end || k0 + 16 <= u.lo ? -1 : p.table[u.n * p.table_stride + (k0 >> p.page_log2)];
        };
        auto held = [&](int b) { return b >= 0 && b < p.num_blocks; };
        int blk = -1, nblk = look_up(u.j0 * KT + lane * 16);
        float ksc = -1.f, vlg = 0.f, vin = 1.f, nks = 0.f, nvs = 0.f;
        auto scales_of = [&]() {
          if (!held(nblk)) return;
          const int64_t at = static_cast<int64_t>(nblk) * p.HKV + u.head;
          nks = p.k_scale[at], nvs = p.v_scale[at];
        };
        scales_of();
        for (int j = u.j0; j < u.j1 && ok; ++j) {
          const int q4 = (j - u.j0) & 3;
          if (q4 == 0) {
            blk = held(nblk) ? nblk : -1;
            ksc = blk >= 0 ? nks : -1.f, vlg = blk >= 0 ? log2f(nvs) : 0.f;
            vin = fabsf(vlg) <= kFarScale ? 1.f / (blk >= 0 ? nvs : 1.f) : NAN;
            nblk = look_up((j + 4) * KT + lane * 16);
          } else if (q4 == 2) {
            scales_of();
          }
          const bool mine = lane / kGroups == q4;
          const uint32_t seen = __ballot_sync(0xffffffffu, mine && blk >= 0);
          const bool leads = mine && blk >= 0 && (seen & page_lanes & ((1u << lane) - 1u)) == 0;
          const int pages = __popc(__ballot_sync(0xffffffffu, leads));
          const int row0 = ((lane % kGroups) & ~(gp - 1)) * 16;  // of my page in the block
          for (int kv = 0; kv < 2; ++kv, ++ic) {
            const int rs = ic % C::NR;
            const uint32_t n = ic / C::NR;
            if (n >= 1 && !(ok = mbar_wait_warp(&bars[RAW_EMPTY0 + rs], (n - 1) & 1, wc, kErrWaitStageEmpty))) break;
            if (kv == 0 && mine) {
              // the block's scales (the ring is deep enough that its last readers are done)
              const uint32_t sr = (ic >> 1) % kScaleRing;
              k_scales[sr * kGroups + lane % kGroups] = ksc;
              v_logs[sr * kGroups + lane % kGroups] = vlg;
              v_invs[sr * kGroups + lane % kGroups] = vin;
            }
            __syncwarp();
            if (lane == 0) {
              if (pages) mbar_arrive_expect_tx(&bars[RAW_FULL0 + rs], (pages * D) << p.page_log2);
              else mbar_arrive(&bars[RAW_FULL0 + rs]);
            }
            __syncwarp();
            if (leads)
              tma_load_4d(sm + C::OFF_RAW + rs * C::RAW + row0 * D, kv ? &maps.v : &maps.k, &bars[RAW_FULL0 + rs], 0,
                          u.head, 0, blk);
          }
        }
      }
      // copies still in flight land before the CTA exits
      if (lane == 0)
        for (uint32_t i = ic > static_cast<uint32_t>(C::NR) ? ic - C::NR : 0u; i < ic; ++i)
          mbar_drain(&bars[RAW_FULL0 + i % C::NR], (i / C::NR) & 1);
      __syncwarp();
    } else if (warp == 9) {
      // ============================================================ MMA issue
      constexpr uint32_t IDESC_S = idesc_f16(false, 128, KT, false, false);
      constexpr uint32_t IDESC_PV = idesc_f16(false, 128, D, false, true);
      const uint32_t sbase = smem_u32(sm), tm = warp_uniform(tmem), elected = elect_lane();
      const uint64_t q_kmaj = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);
      const uint64_t t_kmaj = sdesc_sw128(sbase + C::OFF_T, 16, 1024);
      const uint64_t t_mn = sdesc_sw128(sbase + C::OFF_T, C::SLAB, 1024);
      // Turns taken so far, a bit each: of Q, P and O of tile w (bit w), of the slots.
      // This warp is what the kernel waits for: of 4180 cycles a block (before V scales
      // went into the softmax's exponent, which made it 3 % longer) it waits 900,
      // the products take 2048, the rest is their issue beside a scheduler's softmax
      // and conversion warps.  Hence one body for both tiles (two copies, fetched
      // anew for every block, cost 5 %), the lane elected once (3 %).
      uint32_t q_turn = 0, p_turn = 0, o_turn = 3, k_slot = 0, k_turn = 0, v_slot = 1, v_turn = 0;
      auto next_slot = [](uint32_t* slot, uint32_t* turn) {
        *slot += 2;
        if (*slot >= C::NT) *slot -= C::NT, *turn ^= 1;
      };
      bool ok = true;
      for (uint32_t uc = 0; ok; ++uc) {
        const PrUnit u = next_unit(uc, &ok);
        if (!ok || !u.valid) break;
        if (u.valid == 2 || u.j1 <= u.j0) continue;
        // (lane 0's, so that the compiler takes them, the loop and what is computed in it for uniform)
        const PrTile t0 = tile_of(u, 0, p), t1 = tile_of(u, 1, p);
        const int lo0 = warp_uniform(t0.lo), hi0 = warp_uniform(t0.hi), lo1 = warp_uniform(t1.lo),
                  hi1 = warp_uniform(t1.hi), j0 = warp_uniform(u.j0), j1 = warp_uniform(u.j1);
        // S of block j + 1 goes behind P V of block j, over its P
        for (int j = j0 - 1; j < j1 && ok; ++j) {
          const bool pv = j >= j0, s = j + 1 < j1;
          if (pv && !(ok = mbar_wait_warp(&bars[T_FULL0 + v_slot], v_turn, wc, kErrWaitKV))) break;
#pragma unroll 1
          for (int w = 0; w < 2 && ok; ++w) {
            const int lo = w ? lo1 : lo0, hi = w ? hi1 : hi0;
            const uint32_t ts = tm + C::T_S + w * 128, to = tm + C::T_O + w * D;
            if (pv && lo <= j && j < hi) {
              const uint64_t v = t_mn + sdesc_step(v_slot * C::TILE);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (!(ok = mbar_wait_warp(&bars[P_READY0 + 2 * w + h], p_turn >> w & 1, wc, kErrWaitP))) break;
                if (h == 0 && j == lo) {  // the tile's O: its softmax warps have read the previous unit's
                  if (!(ok = mbar_wait_warp(&bars[O_FREE0 + w], o_turn >> w & 1, wc, kErrWaitDQEmpty))) break;
                  o_turn ^= 1u << w;
                }
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < HK / 16; ++kk)
                  mma_ts_e(to, ts + h * 64 + kk * 8, v + sdesc_step((h * HK / 16 + kk) * 2048), IDESC_PV,
                           j > lo || h > 0 || kk > 0, elected);
                mma_commit_w(&bars[O_DONE0 + 2 * w + h]);
              }
              if (!ok) break;
              p_turn ^= 1u << w;
            }
            if (pv && w == 1) mma_commit_w(&bars[T_EMPTY0 + v_slot]);
            if (s) {
              if (w == 0 && !(ok = mbar_wait_warp(&bars[T_FULL0 + k_slot], k_turn, wc, kErrWaitKV))) break;
              if (lo <= j + 1 && j + 1 < hi) {
                if (j + 1 == lo) {  // the unit's Q
                  if (!(ok = mbar_wait_warp(&bars[Q_FULL0 + w], q_turn >> w & 1, wc, kErrWaitStageFull))) break;
                  q_turn ^= 1u << w;
                }
                tc_fence_after();
                const uint64_t q = q_kmaj + sdesc_step(w * C::QTILE), k = t_kmaj + sdesc_step(k_slot * C::TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                  mma_ss_e(ts, q + sdesc_step((kk / 4) * C::QSLAB + (kk % 4) * 32),
                           k + sdesc_step((kk / 4) * C::SLAB + (kk % 4) * 32), IDESC_S, kk > 0, elected);
                mma_commit_w(&bars[S_FULL0 + w]);
              }
              if (w == 1) mma_commit_w(&bars[T_EMPTY0 + k_slot]);
            }
          }
          if (pv) next_slot(&v_slot, &v_turn);
          if (s) next_slot(&k_slot, &k_turn);
        }
      }
      // every MMA issued by this warp completes before TMEM is released
      mma_commit_w(&bars[DRAIN]);
      if (lane == 0) mbar_drain(&bars[DRAIN], 0);
      __syncwarp();
    }
    // warp 11: nothing to do
    finish();
    return;
  }

  setmaxnreg_inc<REG_SOFT>();
  // ============================================================ softmax of tile w (one row a thread)
  const int w = warp >> 2, quad = warp & 3;
  const int trow = quad * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t tO = tmem + lane_off + C::T_O + w * D;
  uint32_t c = 0, bc = 0;  // blocks of this tile, and of the CTA, over all units so far
  bool ok = true;
  for (uint32_t uc = 0; ok; ++uc) {
    const PrUnit u = next_unit(uc, &ok);
    if (!ok || !u.valid) break;
    if (u.valid == 2) continue;
    const uint32_t bc0 = bc;
    bc += u.j1 - u.j0;
    const PrTile tl = tile_of(u, w, p);
    const int row = u.row0 + w * BQ + trow;  // of the request
    if (u.row0 + w * BQ >= u.R) continue;    // the tile is past the request's rows
    const bool live = row < u.R;
    const int qi = row / p.G, hq = u.head * p.G + row % p.G;
    const int64_t pos = static_cast<int64_t>(u.a) + qi;
    const bool any = tl.lo < tl.hi;
    float rs = 0.f;  // what a raw score is multiplied with, beside its page's scale
    int my_lo = 0, my_hi = 0;
    if (any) {
      // ---- my row of Q in fp16 (the tile's last S products completed before its last softmax block)
      const KvReq r{u.a, u.nq, u.L, u.off, u.R};
      if (live) kv_row_keys(r, qi, p.causal, p.window, &my_lo, &my_hi);
      const uint8_t* const src = p.q + 2 * (pos * p.sq_s + static_cast<int64_t>(hq) * p.sq_h);
      float amax = 0.f;
      uint4 x[D / 8];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (live) x[i] = *reinterpret_cast<const uint4*>(src + 16 * i);
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack2<BF16>(xs[e]);
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      float back;
      const float up = to_top(amax, &back);
      rs = back * p.scale_log2;
      uint8_t* const qt = sm + C::OFF_Q + w * C::QTILE;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack2<BF16>(xs[e]);
          y[e] = pack2<false>(f.x * up, f.y * up);
        }
        *reinterpret_cast<uint4*>(qt + (i / 8) * C::QSLAB + sw128_offset(trow, i % 8)) = make_uint4(y[0], y[1], y[2], y[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Q_FULL0 + w]);
    }
    // The row's weights, their sum l and O are at 2^ref.  (Rows past the request's last one go
    // along with a max of their own.)
    float m_used = live ? -INFINITY : 0.f, l = 0.f, ref = kKvRefNone, most = most_sum(ref);
    for (int jh = 2 * tl.lo; jh < 2 * tl.hi; ++jh) {
      const int h2 = jh & 1, k0 = jh * HK;
      const uint32_t tS = tmem + lane_off + C::T_S + w * 128 + h2 * 64;
      if (h2 == 0) {
        if (!(ok = mbar_wait_warp(&bars[S_FULL0 + w], c & 1, wc, kErrWaitS))) break;
        tc_fence_after();
      }
      uint32_t sr[HK];  // my row's scores (in flight while the scales are looked at)
      tmem_ld32(tS, sr);
      tmem_ld32(tS + 32, sr + 32);
      const float* const sc = k_scales + ((bc0 + (jh >> 1) - u.j0) % kScaleRing) * kGroups + h2 * 4;
      const float4 sa = *reinterpret_cast<const float4*>(sc);
      const float4 sb = *reinterpret_cast<const float4*>(sc + kScaleRing * kGroups);
      const float4 si = *reinterpret_cast<const float4*>(sc + 2 * kScaleRing * kGroups);
      float f[4] = {sa.x, sa.y, sa.z, sa.w};
      bool masked = k0 < tl.all_lo || k0 + HK > tl.all_hi;
#pragma unroll
      for (int g = 0; g < 4; ++g) masked |= f[g] < 0.f;
      uint32_t no_page = 0;  // groups without a page
      if (masked) {
#pragma unroll
        for (int g = 0; g < 4; ++g) no_page |= f[g] < 0.f ? 1u << g : 0u;
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) f[g] = fmaxf(fabsf(f[g]) * rs, 0x1p-126f);  // (0 times -inf would be NaN)
      const int v_lo = my_lo - k0, v_hi = my_hi - k0;
      // One pass with the max at hand, no max taken: while the half block's sums of P
      // and of the weights stay at or below 2^15, none is above it, which fp16 and
      // the f32 sums hold as well as smaller ones.  Past that (or at a row's first
      // key), the max is found and the half computed again (its scores are still
      // there: the weights are stored last).
      const bool first = m_used == -INFINITY;
      float2 sum;  // of P at 2^ref
      bool need = first;  // (row by row, so that no row's result depends on another's)
      {
        uint32_t pw[HK / 2];
        const float base = ref - (first ? 0.f : m_used);
        const float b[4] = {sb.x + base, sb.y + base, sb.z + base, sb.w + base};
        tmem_ld_wait();
        if (__builtin_expect(masked, 0)) {
#pragma unroll
          for (int k = 0; k < HK; ++k)
            if (k < v_lo || k >= v_hi || (no_page >> (k / 16) & 1u)) sr[k] = __float_as_uint(-INFINITY);
        }
        float2 part[4];  // sums of the weights of each group
#pragma unroll
        for (int e = 0; e < HK / 2; ++e) {
          const float fg = f[e / 8], bg = b[e / 8];
          const float2 y = __ffma2_rn(make_float2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])),
                                      make_float2(fg, fg), make_float2(bg, bg));
          const float2 w = make_float2(ex2(y.x), ex2(y.y));
          part[e / 8] = e % 8 == 0 ? w : __fadd2_rn(part[e / 8], w);
          pw[e] = pack2<false>(w.x, w.y);
        }
        const float2 all = __fadd2_rn(__fadd2_rn(part[0], part[1]), __fadd2_rn(part[2], part[3]));
        sum = __fmul2_rn(part[0], make_float2(si.x, si.x));
        sum = __ffma2_rn(part[1], make_float2(si.y, si.y), sum);
        sum = __ffma2_rn(part[2], make_float2(si.z, si.z), sum);
        sum = __ffma2_rn(part[3], make_float2(si.w, si.w), sum);
        need |= !(sum.x + sum.y <= most && all.x + all.y <= kMostSum);
        need &= live;
        if (__builtin_expect(!__any_sync(0xffffffffu, need), 1)) {
#pragma unroll
          for (int h = 0; h < HK / 32; ++h) tmem_st16(tS + h * 16, pw + h * 16);
        }
      }
      if (__builtin_expect(__any_sync(0xffffffffu, need), 0)) {
        auto load_scores = [&](int h, uint32_t* x) {  // 32 scores of the row, -inf where the key is not seen
          tmem_ld32(tS + h * 32, x);
          tmem_ld_wait();
          if (masked) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (h * 32 + k < v_lo || h * 32 + k >= v_hi || (no_page >> (h * 2 + k / 16) & 1u))
                x[k] = __float_as_uint(-INFINITY);
          }
        };
        float m_new = m_used, top = -INFINITY;  // top: log2 of the largest weight here, beside the max
#pragma unroll 1
        for (int h = 0; h < HK / 32; ++h) {
          uint32_t x[32];
          load_scores(h, x);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < 16; ++k) mx = fmaxf(mx, __uint_as_float(x[g * 16 + k]));
            mx *= h == 0 ? f[g] : f[2 + g];
            m_new = fmaxf(m_new, mx);
            top = fmaxf(top, mx + (g == 0 ? (h == 0 ? sb.x : sb.z) : (h == 0 ? sb.y : sb.w)));
          }
        }
        float up = 0.f, now = ref;  // what the max grows by, the row's new ref
        if (need && m_new != -INFINITY) {
          up = first ? 0.f : m_new - m_used;
          // the largest weight: one of these or, as it was where ref was set, an earlier one
          now = weight_ref(kTop, first ? top - m_new : fmaxf(top - m_new, kTop - ref - up));
          m_used = m_new;
        }
        if (__any_sync(0xffffffffu, !first && (up != 0.f || now != ref))) {
          // the tile's previous P V (of this unit: some max is finite) has completed before its O rows are scaled
          if (!(ok = mbar_wait_warp(&bars[O_DONE0 + 2 * w + (h2 ^ 1)], (c - 1 + h2) & 1, wc, kErrWaitDQFull))) break;
          tc_fence_after();
          const float shrink = first ? 1.f : ex2(now - ref - up);
          l *= shrink;
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t r[32];
            tmem_ld32(tO + ch * 32, r);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * shrink);
            tmem_st16(tO + ch * 32, r);
            tmem_st16(tO + ch * 32 + 16, r + 16);
          }
        }
        ref = now, most = most_sum(ref);
        const float msub = m_used == -INFINITY ? 0.f : m_used, base = ref - msub;
        sum = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int h = 0; h < HK / 32; ++h) {
          uint32_t x[32], pw[16];
          load_scores(h, x);
          float2 part[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float fg = h == 0 ? f[g] : f[2 + g];
            const float lv = g == 0 ? (h == 0 ? sb.x : sb.z) : (h == 0 ? sb.y : sb.w);
            float iv = g == 0 ? (h == 0 ? si.x : si.z) : (h == 0 ? si.y : si.w), bg = lv + base, wg = 1.f;
            if (!(iv == iv) || most < 0.f) bg = -msub, wg = weight_factor(lv, ref), iv = ex2(ref);  // P, and the weight as a product
#pragma unroll
            for (int e = 8 * g; e < 8 * g + 8; ++e) {
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])),
                                          make_float2(fg, fg), make_float2(bg, bg));
              const float2 w = make_float2(ex2(y.x), ex2(y.y));
              part[g] = e % 8 == 0 ? w : __fadd2_rn(part[g], w);
              pw[e] = pack2<false>(w.x * wg, w.y * wg);
            }
            sum = __ffma2_rn(part[g], make_float2(iv, iv), sum);
          }
          tmem_st16(tS + h * 16, pw);  // over scores that have been read for good
        }
      }
      l += sum.x + sum.y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[P_READY0 + 2 * w + h2]);
      c += h2;
    }
    if (!ok) break;
    // ---- the row's O and LSE, or its part
    if (any) {
      if (!(ok = mbar_wait_warp(&bars[O_DONE0 + 2 * w + 1], (c - 1) & 1, wc, kErrWaitDQFull))) break;
      tc_fence_after();
    }
    const bool whole = u.slot < 0;
    const int64_t prow = whole ? 0 : static_cast<int64_t>(u.slot) * RT + w * BQ + trow;
    const float back = ex2(-ref), fo = whole ? (l == 0.f ? 0.f : 1.f / l) : back;
    if (live) {
      if (whole) store_lse(p, pos, hq, m_used, l * back);
      else p.part_ml[prow] = make_float2(m_used, l * back);
    }
#pragma unroll 1
    for (int ch = 0; ch < D / 32; ++ch) {
      uint32_t r[32];
      float v[32];
      if (any) {
        tmem_ld32(tO + ch * 32, r);
        tmem_ld_wait();
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = any ? __uint_as_float(r[e]) * fo : 0.f;
      if (live) {
        if (whole) {
          store_o<BF16, 32>(p, pos, hq, ch * 32, v);
        } else {
          float* const to = p.part_o + prow * D + ch * 32;
#pragma unroll
          for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
    }
    if (any) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[O_FREE0 + w]);
    }
  }
  finish();
}

template <int D, bool BF16>
cudaError_t launch_t(const KvAttnParams& p, const KvMaps& maps, int grid, cudaStream_t st) {
  using C = PrCfg<D>;
  auto kern = kv_prompt_kernel<D, BF16>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem_once(kern, C::SMEM, &done);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, grid, THREADS, C::SMEM, st, maps, p);
}

}  // namespace

cudaError_t launch_kv_prompt(const KvAttnParams& p, const KvMaps& maps, bool bf16, int sms, KvJoinPart* left,
                             cudaStream_t st) {
  const int grid = imin(sms, kKvPrMaxCtas);
  *left = kv_join_part(p, grid, grid, 1, RT);
  if (p.D == 64) return bf16 ? launch_t<64, true>(p, maps, grid, st) : launch_t<64, false>(p, maps, grid, st);
  return bf16 ? launch_t<128, true>(p, maps, grid, st) : launch_t<128, false>(p, maps, grid, st);
}

}  // namespace ab
