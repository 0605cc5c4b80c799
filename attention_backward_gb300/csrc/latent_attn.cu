// Attention over latent rows: absorbed queries of 576 columns against rows
// (c | k) that all heads share, whose first 512 columns are the values too
// (include/attn_latent.h).  One kernel body serves the paged cache (single
// tokens, drafted ones, prompts) and the index lists of top-k sparse attention.
//
// A unit is 64 rows (query, head) of a request, or the heads of one token's
// list, with the tiles of 64 keys that they see.  Per tile, with the rows of Q as
// the products' N:
//
//   load    64 latent rows into nine 128-byte-swizzled slabs of 64 columns
//   S^T  = K Q^T          M = 64 keys, N = 64 rows, K = 576
//   P^T  = 2^((S^T - m) scale log2 e + 7)  16 bits, in shared memory
//   O^T += C^T P^T        four M-tiles of 128 latent columns, N = 64, K = 64 keys
//
// so that a tile is read once from memory, serves as K (K-major) and as C^T
// (M-major), and 512 columns of O fit tensor memory beside the scores: rows as M
// would need all of it.  (Fewer rows take the products of 64.)
//
// Softmax: eight warps, a quarter of the keys and half of the rows each; the scores
// arrive as fragments (a thread: 2 keys, 8 rows).  A row's reference m, one of its scores, is
// kept until a weight would pass 2^15: one vote of the warps a tile, and only then is the max
// taken, l scaled and O^T scaled in tensor memory.  The largest weight is then 2^7: fp16
// weights keep their normal range down to 2^-21 of it and steps of 2^-31.  (m is taken off
// before the scaling: of scores from 2^27 on, a scaled m would be rounded by more than fp16's
// room above 2^7.)  l is summed from the f32 weights, a thread's share of the keys in
// registers until the unit ends.
//
// Cache: the line of kv_sched.cuh, cut evenly over the CTAs; a unit split over
// several leaves f32 partials that latent_join.cu joins.  Where requests have more
// than 64 rows two CTAs share a part, 64 rows each of units of 128, so that the second
// reads its keys from L2.  Lists: a unit a token and KV group, longest lists first, or,
// where these are few, parts of their tiles.
//
// Rows are loaded by 16-byte asynchronous copies of four warps, a slab's swizzle written
// by address; rows that are not visible are filled with zeros.  (TMA gathers of four rows
// took 37 ns each, 5.4 us a tile; boxes of 64 rows are as fast as the copies, but
// take 32 ns each whatever their size, and pages of 16 need 36 a tile.)
//
// Bound by DRAM where the rows of a request fit one tile of 64: 64 single tokens of 64 heads
// on 8192 rows 119 us with the join, 5.1 TB/s, 75 % of the copy rate (the stream itself runs
// at 5.9).  Where rows come from L2, the products' reads of shared memory (147 KB for S, 96 for
// O a tile) account for two thirds of a tile's time, at 128 bytes a cycle; the rest is the chain
// from the loads over S and the softmax to O, and S's M of 64, half of the tensor core's rows:
// 4096 lists of up to 2048 rows (1536 on average), 64 heads 0.95 ms, 920 TFLOP/s, 48 % of the
// bf16 peak, the tensor pipe active for 60 % of it.
// One request of 385 rows, 16 heads: 12.7 us with the join, of which 7 start and end the
// kernels.
//
// Warp roles (16 warps): 0-7 softmax and output, 8-11 loads of rows, 12 of Q, 13 issue
// of the scores, 14 the walk, a unit ahead of the others, 15 issue of O.  Every wait is
// bounded.
#include <cmath>

#include "cvt.cuh"
#include "kv_launch.h"
#include "kv_sched.cuh"
#include "latent.h"
#include "latent_issue.cuh"
#include "sm103.cuh"

namespace ab {

namespace {

constexpr int NR = kLatRows, KT = kLatKeys;
constexpr int NSLAB = kLatRow / 64;
constexpr int SLAB = KT * 128;  // [64 rows x 64 columns] 16-bit, 128-byte swizzled
constexpr int TILE = NSLAB * SLAB;
constexpr int STAGES = 2;
// A stage is loaded and freed in five groups: the two slabs of each M-tile of O, and the
// key part, whose slab takes P once the scores are made.
constexpr int GROUPS = 5;
constexpr int kWarps = 16, THREADS = kWarps * 32;
constexpr int SOFT = 256;  // threads of the softmax warps
constexpr float kTop = kLatTop, kMost = 15.f;  // log2 of a row's largest weight when its max is taken, and of the most it may grow to
constexpr float kNone = -3.402823466e38f;  // reference of a row that has seen no key, the least that one may have

enum LatBar : int {
  Q_FULL = 0,                // the loading warp (lists: a copy)
  Q_EMPTY,                   // every S of the unit has completed
  FULL0,                     // per stage and group of slabs
  EMPTY0 = FULL0 + STAGES * GROUPS,  // the same: its last products have completed
  S_FULL0 = EMPTY0 + STAGES * GROUPS,  // per score buffer
  P_READY0 = S_FULL0 + 2,    // tiles in turn: the softmax warps
  O_DONE0 = P_READY0 + 2,    // tiles in turn: its O products, and all before them
  O_FREE = O_DONE0 + 2,      // the softmax warps read the unit's O
  UNIT_FULL0,                // 2 slots
  UNIT_EMPTY0 = UNIT_FULL0 + 2,  // 15 warps
  DRAIN0 = UNIT_EMPTY0 + 2,  // of the issuing warps
  NUM_BARS = DRAIN0 + 2
};
// Arrivals that complete barrier i.
__device__ __forceinline__ int arrivals(int i) {
  // every copying thread; of the last group also a lane a warp, for the bits
  if (i >= FULL0 && i < EMPTY0) return (i - FULL0) % GROUPS == GROUPS - 1 ? 132 : 128;
  if (i == O_FREE || (i >= P_READY0 && i < O_DONE0)) return SOFT / 32;
  return i >= UNIT_EMPTY0 && i < DRAIN0 ? 15 : 1;
}

// A unit, or the CTA's part of one: key tiles [j0, j1).
struct LatUnit {
  int valid;  // 0: no more, 1: work, 2: nothing to do
  int n;      // request, or batch row
  int a, nq, L, off;  // first token of q, queries, visible positions, key position of query 0 (lists: a = token)
  int row0, live;     // first row in the request (lists: first head), rows of this CTA
  int j0, j1;
  int slot;  // -1: the whole unit, else the slot of its partial rows
};

// A place on the line: request, row tile, position in it.
struct LatCursor {
  int n, rt, pos;
  KvReq r;
};

struct LatShared {
  int64_t row[NR];    // a row's place in o
  float mx[4][NR];    // per quarter of the keys and row: a max, or a sum
  float f[NR];        // per row: a factor
  float ref[NR];
  int hi[NR];         // keys that a row sees
  LatUnit units[2];
  uint32_t bits[STAGES][4];  // of a stage's tile and 16-key group: its keys that are held, and visible if the mask leaves them
  uint64_t bars[NUM_BARS];
  int64_t work[kWarps];  // line positions of each warp's requests
  LatCursor cursor;
  uint32_t tmem;
  int abort;
};

constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + TILE;
constexpr int OFF_SH = OFF_K + STAGES * TILE;
__device__ __forceinline__ int p_at(uint32_t stage) { return OFF_K + stage * TILE + (NSLAB - 1) * SLAB; }
constexpr int SMEM = OFF_SH + static_cast<int>(sizeof(LatShared));
static_assert(SMEM <= 227 * 1024, "shared memory budget");

constexpr uint32_t T_S = 0, T_O = 128;  // score buffers at 0 and 64; O^T tile m at 128 + 64 m

// A value that all lanes have, as one the compiler knows to be the warp's.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }

// 16 lanes x 32 columns of a warp's quarter as fragments: registers 4 j + (0, 1) are
// row lane / 4, columns 8 j + 2 (lane % 4) + (0, 1); 4 j + (2, 3) row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, uint32_t bytes) {  // the rest reads zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// The softmax warps; true in all of them if it is in one.
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 2, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 2, 256;" ::: "memory"); }

// Of 8 values in each of the lanes l, l ^ 4, l ^ 8, .. (8 of them), the one of column
// column_of(lane) over all 8.
__device__ __forceinline__ int column_of(int lane) { return (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1); }
template <typename F>
__device__ __forceinline__ float reduce8(float (&v)[8], int lane, F f) {
#pragma unroll
  for (int n = 4, o = 16; n > 0; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = f(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return v[0];
}

// ---------------------------------------------------------------- the line

template <int RT>
__device__ __forceinline__ int tile_work(const KvReq& r, int rt, const KvAttnParams& p) {
  return kv_row_tile<RT, KT>(r, rt, p).n + kLatCost;
}

// Positions of a request, all lanes together.
template <int RT>
__device__ __forceinline__ int64_t lanes_work(const KvAttnParams& p, const KvReq& r) {
  int64_t w = 0;
  const int nt = kv_row_tiles<RT>(r);
  for (int rt = threadIdx.x & 31; rt < nt; rt += 32) w += tile_work<RT>(r, rt, p);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  return w;
}

__device__ __forceinline__ int64_t lanes_scan(int64_t w) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += v;
  }
  return w;
}

__device__ __forceinline__ KvReq from_lane(const KvReq& r, int src) {
  return {__shfl_sync(0xffffffffu, r.a, src), __shfl_sync(0xffffffffu, r.nq, src), __shfl_sync(0xffffffffu, r.L, src),
          __shfl_sync(0xffffffffu, r.off, src), __shfl_sync(0xffffffffu, r.R, src)};
}

// Each thread has ``per`` requests in a row: their positions, and the last of them.
template <int RT>
__device__ __forceinline__ int64_t thread_work(const KvAttnParams& p, int per, KvReq* last) {
  const int lane = threadIdx.x & 31;
  int64_t w = 0;
  for (int k = 0; k < per; ++k) {
    const int n = threadIdx.x * per + k;
    KvReq r{};
    if (n < p.N) r = kv_request(n, p);
    if (r.R > 0 && r.R <= RT) w += tile_work<RT>(r, 0, p);
    for (uint32_t m = __ballot_sync(0xffffffffu, r.R > RT); m != 0; m &= m - 1) {  // of several row tiles
      const int src = __ffs(m) - 1;
      const int64_t all = lanes_work<RT>(p, from_lane(r, src));
      if (lane == src) w += all;
    }
    *last = r;
  }
  return w;
}

// The cursor of position x, which lies x positions behind the start of the requests
// [n0, n0 + per) and within them (one warp); r: the last of them.
template <int RT>
__device__ __forceinline__ LatCursor find(const KvAttnParams& p, int n0, int per, KvReq r, int64_t x) {
  const int lane = threadIdx.x & 31;
  LatCursor c{n0 + per - 1, 0, 0, {}};
  for (int k = 0; k + 1 < per; ++k) {
    const KvReq q = kv_request(n0 + k, p);
    const int64_t w = lanes_work<RT>(p, q);
    if (x < w) {
      c.n = n0 + k, r = q;
      break;
    }
    x -= w;
  }
  c.r = r;
  const int nt = kv_row_tiles<RT>(r);
  for (int b = 0; b < nt; b += 32) {
    const int64_t w = b + lane < nt ? tile_work<RT>(r, b + lane, p) : 0;
    const int64_t inc = lanes_scan(w);
    const uint32_t past = __ballot_sync(0xffffffffu, x < inc);
    if (past == 0) {
      x -= __shfl_sync(0xffffffffu, inc, 31);
      continue;
    }
    const int src = __ffs(past) - 1;
    c.rt = b + src;
    c.pos = static_cast<int>(x - __shfl_sync(0xffffffffu, inc - w, src));
    break;
  }
  return c;
}

// GROUP: CTAs that share a part of the line; 0: index lists.
template <int GROUP, bool BF16>
__global__ void __launch_bounds__(THREADS, 1)
    latent_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ LatParams lp) {  // map: of Q
  constexpr bool LISTS = GROUP == 0;
  constexpr int RT = NR * (LISTS ? 1 : GROUP);
  const KvAttnParams& p = lp.a;
  extern __shared__ __align__(1024) uint8_t sm[];
  LatShared& sh = *reinterpret_cast<LatShared*>(sm + OFF_SH);
  uint64_t* const bars = sh.bars;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---------------------------------------------------------------- set-up, beside the end of the launch before
  if (warp == 12) {
    for (int i = lane; i < NUM_BARS; i += 32) mbar_init(&bars[i], arrivals(i));
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  // (the join's blocks, let in at once, wait beside the last parts and slow them: 300 requests of
  // 300 rows 40 -> 43 us, 64 of 4000 67 -> 68.5)
  grid_dependency_wait();
  volatile int* const abort_flag = &sh.abort;
  const WaitCtx wc{abort_flag, LISTS ? p.err : p.cta_err + blockIdx.x, p.timeout_ns};
  // a unit lasts as long as its keys do: waits for one to begin or to be taken
  // have a limit of their own (any wait that runs out ends the others too)
  const WaitCtx wu{abort_flag, wc.err, 64 * p.timeout_ns};
  const bool aligned = (smem_u32(sm) & 1023u) == 0;
  if (threadIdx.x == 0) {
    if (LISTS) {
      // (the call's error word, which a wait sets after a second at the earliest)
      if (blockIdx.x == 0) *p.err = aligned ? kErrNone : kErrAlign;
    } else {
      *wc.err = aligned ? kErrNone : kErrAlign;
      p.desc[blockIdx.x] = make_int4(0, 0, 0, -1);
    }
    sh.abort = 0;
  }
  // ---------------------------------------------------------------- the CTA's part of the line
  int64_t total = 0, begin = 0, end = 0;
  int parts = 1, per = 0;
  int64_t mine = 0, upto = 0;  // positions of my requests, and up to their end
  const int part = LISTS ? 0 : blockIdx.x / imax(GROUP, 1), sub = LISTS ? 0 : blockIdx.x % imax(GROUP, 1);
  KvReq last{};
  if constexpr (!LISTS) {
    per = (p.N + THREADS - 1) / THREADS;
    mine = thread_work<RT>(p, per, &last);
    upto = lanes_scan(mine);
    if (lane == 31) sh.work[warp] = upto;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  auto leave = [&]() {  // (all threads do)
    if (warp == 13) tmem_dealloc(tmem, 512);
  };
  if (!aligned) return leave();
  if constexpr (!LISTS) {
    int64_t before = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int64_t w = sh.work[i];
      if (i < warp) before += w;
      total += w;
    }
    if (total == 0) return leave();
    upto += before;
    const int64_t want = (total + kLatMinWork - 1) / kLatMinWork;
    const int most = gridDim.x / GROUP;
    parts = want < most ? static_cast<int>(want) : most;
    if (part >= parts) return leave();
    begin = kv_part_begin(total, part, parts), end = kv_part_begin(total, part + 1, parts);
    // the warp whose requests hold the first position looks it up
    const uint32_t here = __ballot_sync(0xffffffffu, begin >= upto - mine && begin < upto);
    if (here != 0) {
      const int src = __ffs(here) - 1;
      const LatCursor c = find<RT>(p, (threadIdx.x - lane + src) * per, per, from_lane(last, src), begin - __shfl_sync(0xffffffffu, upto - mine, src));
      if (lane == 0) sh.cursor = c;
    }
  }

  __syncthreads();

  // the uc-th unit of this CTA
  auto next_unit = [&](uint32_t uc, bool* okp) -> LatUnit {
    const uint32_t slot = uc & 1;
    LatUnit u{};
    if (!(*okp = mbar_wait_warp(&bars[UNIT_FULL0 + slot], (uc >> 1) & 1, wu, kErrWaitTile))) return u;
    u = sh.units[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[UNIT_EMPTY0 + slot]);
    return u;
  };

  // the same of a lane alone: its units with tiles
  auto next_tiles = [&](uint32_t* uc, int* tiles) -> bool {
    for (;; ++*uc) {
      const uint32_t slot = *uc & 1;
      if (!mbar_wait(&bars[UNIT_FULL0 + slot], (*uc >> 1) & 1, wu, kErrWaitTile)) return false;
      const int valid = sh.units[slot].valid;
      *tiles = sh.units[slot].j1 - sh.units[slot].j0;
      mbar_arrive(&bars[UNIT_EMPTY0 + slot]);
      if (!valid) return false;
      if (valid != 2 && *tiles > 0) return ++*uc, true;
    }
  };

  if (warp == 14) {
    // ============================================================ the walk
    auto publish = [&](uint32_t uc, const LatUnit& u) -> bool {
      const uint32_t slot = uc & 1;
      if (uc >= 2 && !mbar_wait_warp(&bars[UNIT_EMPTY0 + slot], ((uc >> 1) - 1) & 1, wu, kErrWaitTile)) return false;
      if (lane == 0) {
        sh.units[slot] = u;
        mbar_arrive(&bars[UNIT_FULL0 + slot]);
      }
      return true;
    };
    if constexpr (LISTS) {
      const int units = lp.B * lp.S * lp.HKV * lp.splits;
      uint32_t uc = 0;
      for (int i = blockIdx.x;; i += gridDim.x, ++uc) {
        LatUnit u{};
        u.valid = i < units;
        if (u.valid) {
          const LatListUnit v = list_unit(i / lp.splits, lp);
          u.n = v.b, u.a = v.t, u.row0 = v.g * lp.gh, u.live = lp.gh;
          const int* const il = lp.idx + v.b * lp.si_b + v.t * lp.si_s + v.g * lp.si_h;
          int last = -1;  // the last entry that lists a row: from the end, 256 at a time
          for (int s0 = (lp.topk - 1) & ~255; s0 >= 0 && last < 0; s0 -= 256) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int s = s0 + 32 * k + lane, j = s < lp.topk ? il[s] : -1;
              if (j >= 0 && j < lp.SKV) last = s;
            }
            last = __reduce_max_sync(0xffffffffu, last);
          }
          const int n = last < 0 ? 0 : last / KT + 1, part = i % lp.splits;
          u.j0 = static_cast<int>(static_cast<int64_t>(n) * part / lp.splits);
          u.j1 = static_cast<int>(static_cast<int64_t>(n) * (part + 1) / lp.splits);
          u.slot = lp.splits > 1 ? i : -1;
        }
        if (!publish(uc, u) || !u.valid) break;
      }
    } else {
      LatCursor cur = sh.cursor;
      KvReq rq = cur.r;
      int64_t x = begin;
      for (uint32_t uc = 0;; ++uc) {
        LatUnit u{};
        int64_t stop = x;
        u.valid = x < end;
        if (u.valid) {
          const KvTiles kt = kv_row_tile<RT, KT>(rq, cur.rt, p);
          const int64_t unit0 = x - cur.pos;
          stop = unit0 + kLatCost + kt.n < end ? unit0 + kLatCost + kt.n : end;
          const int part0 = imax(0, cur.pos - kLatCost), part1 = imax(0, static_cast<int>(stop - unit0) - kLatCost);
          const bool whole = part0 == 0 && part1 == kt.n;
          u.n = cur.n, u.a = rq.a, u.nq = rq.nq, u.L = rq.L, u.off = rq.off;
          u.row0 = cur.rt * RT + sub * NR, u.live = imin(NR, rq.R - u.row0);
          u.j0 = kt.t0 + part0;
          u.j1 = kt.hi > kt.lo ? kt.t0 + part1 : u.j0;  // (a unit that sees nothing has no tile)
          u.slot = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (part0 > 0 ? 0 : 1);
          if (part1 <= part0 || u.live <= 0) u.valid = 2;  // only start-up positions, or no rows: nothing to do
          if (lane == 0 && part0 > 0 && part1 == kt.n && u.live > 0)
            p.desc[blockIdx.x] = make_int4(rq.a, u.row0, u.live, kv_part_of(total, unit0 + kLatCost, parts));
        }
        if (!publish(uc, u) || !u.valid) break;
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
  } else if (warp == 12) {
    // ============================================================ Q
    uint32_t qc = 0;
    bool ok = true, copied = false;
    for (uint32_t uc = 0; ok; ++uc) {
      const LatUnit u = next_unit(uc, &ok);
      if (!ok || !u.valid) break;
      if (u.valid == 2 || u.j1 <= u.j0) continue;
      // every S of the unit before, which lasts as long as that unit
      if (qc >= 1 && !(ok = mbar_wait_warp(&bars[Q_EMPTY], (qc - 1) & 1, wu, kErrWaitStageEmpty))) break;
      ++qc;
      if (LISTS || p.q == nullptr) {
        // lists: 64 heads of the token; else 64 rows of [T * H, 576].  (Those past the
        // unit's may be anything: they are columns of the products of their own.)
        if (lane == 0) mbar_arrive_expect_tx(&bars[Q_FULL], TILE);
        __syncwarp();
        if (lane < NSLAB)
          tma_load_4d(sm + OFF_Q + lane * SLAB, &map, &bars[Q_FULL], lane * 64, LISTS ? u.row0 : u.a * p.G + u.row0,
                      LISTS ? u.a : 0, LISTS ? u.n : 0);
        copied = true;
      } else {
        const int r = lane >> 3, c = lane & 7;  // four rows at once, 128 bytes each
#pragma unroll 2
        for (int at = r; at < NR; at += 4) {
          const int row = u.row0 + at;
          const bool on = at < u.live;
          const uint8_t* src = p.q;
          if (on) src += 2 * (static_cast<int64_t>(u.a + row / p.G) * p.sq_s + (row % p.G) * p.sq_h + 8 * c);
          const uint32_t dst = smem_u32(sm + OFF_Q) + sw128_offset(at, c);
#pragma unroll
          for (int s = 0; s < NSLAB; ++s) copy16_async(dst + s * SLAB, on ? src + s * 128 : src, on ? 16 : 0);
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Q_FULL]);
      }
    }
    if (copied && lane == 0) mbar_drain(&bars[Q_FULL], (qc - 1) & 1);  // a copy in flight lands before the CTA exits
    __syncwarp();
  } else if (warp == 13) {
    // ============================================================ scores
    // (O has a warp of its own: the products are so short that their issue counts, and
    // neither warp waits on what the other is waiting for.  One lane does all of it, as a wait
    // of the whole warp takes 70 to 140 cycles: 2048 lists of 1024 rows, 64 heads 356 -> 338 us.
    // O's by one lane, whose waits are few, make that 351.)
    if (elect_lane()) {
      constexpr uint32_t IDESC = idesc_f16(BF16, KT, NR, false, false);
      const uint64_t k_kmaj = sdesc_sw128(smem_u32(sm) + OFF_K, 16, 1024);
      const uint64_t q_kmaj = sdesc_sw128(smem_u32(sm) + OFF_Q, 16, 1024);
      uint32_t kc = 0, qc = 0, uc = 0;
      int tiles;
      bool ok = true;
      while (ok && next_tiles(&uc, &tiles)) {
        if (!(ok = mbar_wait(&bars[Q_FULL], qc & 1, wc, kErrWaitStageFull))) break;
        ++qc;
        for (const uint32_t end = kc + tiles; kc < end; ++kc) {
          const uint32_t st = kc % STAGES, phase = (kc / STAGES) & 1, d = tmem + T_S + 64 * (kc & 1);
          // the softmax has read the scores of two tiles ago
          if (kc >= 2 && !(ok = mbar_wait(&bars[P_READY0 + (kc & 1)], ((kc >> 1) - 1) & 1, wc, kErrWaitSFree))) break;
          const uint64_t a = k_kmaj + sdesc_step(st * TILE);
#pragma unroll
          for (int g = 0; g < GROUPS; ++g) {
            if (!(ok = mbar_wait(&bars[FULL0 + st * GROUPS + g], phase, wc, kErrWaitKV))) break;
            fence_proxy_async_smem();  // (the copies are the generic proxy's)
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < (g < 4 ? 8 : 4); ++kk) {
              const uint64_t o = sdesc_step((2 * g + kk / 4) * SLAB + kk % 4 * 32);
              mma_ss_e(d, a + o, q_kmaj + o, IDESC, g + kk > 0, 1u);
            }
          }
          if (!ok) break;
          mma_commit_1(&bars[S_FULL0 + (kc & 1)]);
        }
        mma_commit_1(&bars[Q_EMPTY]);
      }
      // every product issued here completes before tensor memory is released
      mma_commit_1(&bars[DRAIN0]);
      mbar_drain(&bars[DRAIN0], 0);
    }
    __syncwarp();
  } else if (warp == 15) {
    // ============================================================ O
    constexpr uint32_t IDESC = idesc_f16(BF16, 128, NR, true, true);
    const uint64_t c_mn = sdesc_sw128(smem_u32(sm) + OFF_K, SLAB, 1024);
    const uint64_t p_mn = sdesc_sw128(smem_u32(sm) + p_at(0), 0, 1024);
    const uint32_t one = elect_lane();
    uint32_t kc = 0, oc = 0;
    bool ok = true;
    for (uint32_t uc = 0; ok; ++uc) {
      const LatUnit u = next_unit(uc, &ok);
      if (!ok || !u.valid) break;
      if (u.valid == 2 || u.j1 <= u.j0) continue;
      // the softmax warps have read the O of the unit before
      if (oc >= 1 && !(ok = mbar_wait_warp(&bars[O_FREE], (oc - 1) & 1, wu, kErrWaitDQEmpty))) break;
      ++oc;
      const uint32_t first = kc;
      for (const uint32_t end = kc + uniform(u.j1 - u.j0); kc < end; ++kc) {
        const uint32_t st = kc % STAGES;
        if (!(ok = mbar_wait_warp(&bars[P_READY0 + (kc & 1)], (kc >> 1) & 1, wu, kErrWaitP))) break;
        tc_fence_after();
        const uint64_t c = c_mn + sdesc_step(st * TILE), pp = p_mn + sdesc_step(st * TILE);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_e(tmem + T_O + 64 * m, c + sdesc_step(2 * m * SLAB + kk * 2048), pp + sdesc_step(kk * 2048), IDESC,
                     kc != first || kk > 0, one);
          mma_commit_w(&bars[EMPTY0 + st * GROUPS + m]);
        }
        mma_commit_w(&bars[EMPTY0 + st * GROUPS + GROUPS - 1]);
        mma_commit_w(&bars[O_DONE0 + (kc & 1)]);
      }
    }
    mma_commit_w(&bars[DRAIN0 + 1]);
    if (lane == 0) mbar_drain(&bars[DRAIN0 + 1], 0);
    __syncwarp();
  } else if (warp >= 8 && warp < 12) {
    // ============================================================ rows: 16 of a tile a warp
    // Eight lanes copy 128 bytes of a row, a warp four rows of a slab at once; a barrier
    // counts the copies' completion itself.  Lanes look up rows a tile ahead.
    const int w = warp - 8, r = lane >> 3, c = lane & 7;
    uint32_t kc = 0;
    bool ok = true;
    for (uint32_t uc = 0; ok; ++uc) {
      const LatUnit u = next_unit(uc, &ok);
      if (!ok || !u.valid) break;
      if (u.valid == 2) continue;
      const int g = LISTS ? u.row0 / lp.gh : 0;
      const int* const list = LISTS ? lp.idx + u.n * lp.si_b + static_cast<int64_t>(u.a) * lp.si_s + g * lp.si_h
                                    : p.table + static_cast<int64_t>(u.n) * p.table_stride;
      auto look_up = [&](int j) {  // a row of the cache, or of the batch row's; -1: none
        const int k = j * KT + 16 * w + (lane & 15);
        if constexpr (LISTS) {
          const int i = j < u.j1 && k < lp.topk ? list[k] : -1;
          return i >= 0 && i < lp.SKV ? i : -1;
        } else {
          const int page = j < u.j1 && k < u.L ? list[k >> p.page_log2] : -1;
          return page >= 0 && page < p.num_blocks ? (page << p.page_log2) + (k & ((1 << p.page_log2) - 1)) : -1;
        }
      };
      int next = look_up(u.j0);
      for (int j = u.j0; j < u.j1; ++j, ++kc) {
        const int st = kc % STAGES;
        const uint32_t n = kc / STAGES;
        const int row = next;
        next = look_up(j + 1);
        const uint32_t held = __ballot_sync(0xffffffffu, row >= 0) & 0xffffu;
        const uint8_t* src[4];
        uint32_t dst[4], bytes[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // my rows 4 i + r
          const int at = __shfl_sync(0xffffffffu, row, 4 * i + r);
          const int64_t line = LISTS ? (static_cast<int64_t>(u.n) * lp.SKV + at) * lp.HKV + g : at;
          src[i] = lp.rows + (at < 0 ? 0 : 2 * (line * lp.row_stride + 8 * c));
          dst[i] = smem_u32(sm + OFF_K + st * TILE) + sw128_offset(16 * w + 4 * i + r, c);
          bytes[i] = at < 0 ? 0u : 16u;
        }
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) {
          uint64_t* const full = &bars[FULL0 + st * GROUPS + k];
          if (n >= 1 && !(ok = mbar_wait_warp(&bars[EMPTY0 + st * GROUPS + k], (n - 1) & 1, wc, kErrWaitStageEmpty))) break;
          if (k == GROUPS - 1 && lane == 0) {
            sh.bits[st][w] = held;
            mbar_arrive(full);
          }
#pragma unroll
          for (int s = 2 * k; s < (k < 4 ? 2 * k + 2 : NSLAB); ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) copy16_async(dst[i] + s * SLAB, bytes[i] ? src[i] + s * 128 : lp.rows, bytes[i]);
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full)) : "memory");
        }
        if (!ok) break;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // copies in flight land before the CTA exits
  } else if (warp < 8) {
    // ============================================================ softmax and output
    const int tid = threadIdx.x, w4 = warp & 3, half = warp >> 2;
    const int ka = 16 * w4 + (lane >> 2);             // my keys: ka, ka + 8
    const int c0 = 32 * half + 2 * (lane & 3);        // my rows: c0 + 8 j + (0, 1), j < 4
    const int mine = column_of(lane), cm = c0 + 8 * (mine >> 1) + (mine & 1);  // the row that reduce8 leaves me
    const uint32_t quarter = static_cast<uint32_t>(w4 * 32) << 16;
    const uint32_t bit_a = 1u << (ka & 15), bit_b = bit_a << 8;  // of group w4
    const auto larger = [](float x, float y) { return fmaxf(x, y); };
    uint32_t kc = 0;
    // The warps meet at named barriers, which have no limit: a warp whose wait ran out
    // goes on (its results are void) to the next vote, where all leave.
    bool bad = false, dead = false;
    auto wait = [&](int bar, uint32_t parity, int code) { bad |= !mbar_wait_warp(&bars[bar], parity, wc, code); };
    for (uint32_t uc = 0; !dead; ++uc) {
      bool got;
      const LatUnit u = next_unit(uc, &got);
      bad |= !got;
      if (softmax_any(bad) || !u.valid) break;
      if (u.valid == 2) continue;
      int hi_all = 0x7fffffff;  // keys that every row sees
      if constexpr (!LISTS) {
        const KvReq r{u.a, u.nq, u.L, u.off, 0};
        int lo;
        kv_row_keys(r, u.row0 / p.G, p.causal, 0, &lo, &hi_all);
        if (tid < NR) kv_row_keys(r, (u.row0 + imin(tid, u.live - 1)) / p.G, p.causal, 0, &lo, &sh.hi[tid]);
      }
      if (tid < NR) {
        sh.ref[tid] = kNone;
        const int row = u.row0 + imin(tid, u.live - 1);
        sh.row[tid] = LISTS ? u.n * lp.so_b + u.a * p.so_s + row * p.so_h
                            : static_cast<int64_t>(u.a + row / p.G) * p.so_s + (row % p.G) * p.so_h;
      }
      float neg[8], l[8];  // minus the references
#pragma unroll
      for (int i = 0; i < 8; ++i) neg[i] = -kNone, l[i] = 0.f;
      softmax_sync();
      for (int j = u.j0; j < u.j1; ++j, ++kc) {
        const int st = kc % STAGES;
        wait(FULL0 + st * GROUPS + GROUPS - 1, (kc / STAGES) & 1, kErrWaitKV);  // (for its bits)
        const uint32_t b0 = sh.bits[st][0], b1 = sh.bits[st][1], b2 = sh.bits[st][2], b3 = sh.bits[st][3];
        wait(S_FULL0 + (kc & 1), (kc >> 1) & 1, kErrWaitS);
        tc_fence_after();
        float s[16];  // 4 j + (0, 1): key ka, rows c0 + 8 j + (0, 1); 4 j + (2, 3): key ka + 8
        tmem_ld_frag32(tmem + quarter + T_S + 64 * (kc & 1) + 32 * half, reinterpret_cast<uint32_t*>(s));
        tmem_ld_wait();
        if ((b0 & b1 & b2 & b3) != 0xffffu || (j + 1) * KT > hi_all) {
          const uint32_t w = sh.bits[st][w4];
          const bool va = w & bit_a, vb = w & bit_b;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int h = LISTS ? 0x7fffffff : sh.hi[c0 + 8 * (i >> 1) + (i & 1)];
            float& x = s[4 * (i >> 1) + (i & 1)];
            float& y = s[4 * (i >> 1) + 2 + (i & 1)];
            if (!va || j * KT + ka >= h) x = -INFINITY;
            if (!vb || j * KT + ka + 8 >= h) y = -INFINITY;
          }
        }
        float top[8], over = -INFINITY;  // over: my largest score, above its row's reference
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          top[i] = fmaxf(s[4 * (i >> 1) + (i & 1)], s[4 * (i >> 1) + 2 + (i & 1)]);
          over = fmaxf(over, top[i] + neg[i]);
        }
        if (softmax_any(fmaf(over, p.scale_log2, kTop) > kMost || bad)) {
          // ---- some row's weights outgrow the type: new references for those
          sh.mx[w4][cm] = reduce8(top, lane, larger);
          if ((dead = softmax_any(bad))) break;
          if (tid < NR) {
            const float m = fmaxf(fmaxf(sh.mx[0][tid], sh.mx[1][tid]), fmaxf(sh.mx[2][tid], sh.mx[3][tid]));
            const float old = sh.ref[tid];
            const bool grown = fmaf(m - old, p.scale_log2, kTop) > kMost;
            sh.f[tid] = grown ? ex2((old - m) * p.scale_log2) : 1.f;
            if (grown) sh.ref[tid] = m;
          }
          softmax_sync();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = c0 + 8 * (i >> 1) + (i & 1);
            neg[i] = -sh.ref[row];
            l[i] *= sh.f[row];
          }
          if (j > u.j0) {
            // O^T of the tiles so far, once their products have completed
            wait(O_DONE0 + ((kc - 1) & 1), ((kc - 1) >> 1) & 1, kErrWaitDQFull);
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
              const uint32_t at = tmem + quarter + T_O + 128 * half + 32 * h;
              const float* const f = sh.f + 32 * (h & 1);
              uint32_t r[32];
              tmem_ld32(at, r);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f[e]);
              tmem_st16(at, r);
              tmem_st16(at + 16, r + 16);
            }
            tmem_st_wait();
          }
        }
        uint8_t* const pt = sm + p_at(st);  // (in place of the key part, which the scores have used)
        const float2 scale2 = make_float2(p.scale_log2, p.scale_log2), top2 = make_float2(kTop, kTop);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 neg2 = make_float2(neg[i], neg[i + 1]);
          const float2 x = __ffma2_rn(__fadd2_rn(make_float2(s[2 * i], s[2 * i + 1]), neg2), scale2, top2);
          const float2 y = __ffma2_rn(__fadd2_rn(make_float2(s[2 * i + 2], s[2 * i + 3]), neg2), scale2, top2);
          const float x0 = ex2(x.x), x1 = ex2(x.y), y0 = ex2(y.x), y1 = ex2(y.y);
          l[i] += x0 + y0, l[i + 1] += x1 + y1;
          const uint32_t at = 4 * half + i / 2;  // 16-byte piece of a key's 64 weights
          *reinterpret_cast<uint32_t*>(pt + sw128_offset(ka, at) + 4 * (lane & 3)) = pack2<BF16>(x0, x1);
          *reinterpret_cast<uint32_t*>(pt + sw128_offset(ka + 8, at) + 4 * (lane & 3)) = pack2<BF16>(y0, y1);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[P_READY0 + (kc & 1)]);
      }
      if (dead) break;
      // ---- the rows' sums, then O
      const bool had = u.j1 > u.j0;
      sh.mx[w4][cm] = reduce8(l, lane, [](float x, float y) { return x + y; });
      softmax_sync();
      if (tid < NR) {
        const float sum = (sh.mx[0][tid] + sh.mx[1][tid]) + (sh.mx[2][tid] + sh.mx[3][tid]);
        const float m = sh.ref[tid];
        sh.f[tid] = sum == 0.f ? 0.f : 1.f / sum;
        if (tid < u.live) {
          if (u.slot < 0) {
            const int row = u.row0 + tid;
            float* const lse = LISTS ? p.lse + (u.n * lp.sl_b + row * p.sl_h + u.a * p.sl_s)
                                     : p.lse + ((row % p.G) * p.sl_h + static_cast<int64_t>(u.a + row / p.G) * p.sl_s);
            *lse = sum == 0.f ? -INFINITY : (fmaf(m, p.scale_log2, -kTop) + log2f(sum)) * 0.69314718055994531f;
          } else {
            p.part_ml[static_cast<int64_t>(u.slot) * NR + tid] = make_float2(m, sum);
          }
        }
      }
      softmax_sync();
      if (had) {
        wait(O_DONE0 + ((kc - 1) & 1), ((kc - 1) >> 1) & 1, kErrWaitDQFull);
        tc_fence_after();
      }
      // my 32 latent columns of two M-tiles, 32 rows at once
#pragma unroll 1
      for (int h = 0; h < 4; ++h) {
        const int d = 256 * half + 128 * (h >> 1) + 32 * w4 + lane, r0 = 32 * (h & 1);
        if (r0 >= u.live) continue;
        uint32_t r[32];
        if (had) {
          tmem_ld32(tmem + quarter + T_O + 128 * half + 32 * h, r);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = 0u;
        }
        const int n = imin(32, u.live - r0);
        if (u.slot >= 0) {
          float* const out = p.part_o + (static_cast<int64_t>(u.slot) * NR + r0) * kLatDim + d;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e < n) out[e * kLatDim] = __uint_as_float(r[e]);
        } else {
          // neighbouring lanes swap, so that each stores two columns of one row of a pair
          uint8_t* const out = p.o + 2 * (d & ~1);
          const int64_t* const at = sh.row + r0 + (lane & 1);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 f = *reinterpret_cast<const float2*>(sh.f + r0 + e);
            const uint32_t w = pack2<BF16>(__uint_as_float(r[e]) * f.x, __uint_as_float(r[e + 1]) * f.y);  // rows e, e + 1
            const uint32_t z = __shfl_xor_sync(0xffffffffu, w, 1);
            const uint32_t y = lane & 1 ? __byte_perm(z, w, 0x7632) : __byte_perm(w, z, 0x5410);
            if (e + (lane & 1) < n) *reinterpret_cast<uint32_t*>(out + 2 * at[e]) = y;
          }
        }
      }
      if (had) {
        // this unit's O is read: the next unit's first products may overwrite it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[O_FREE]);
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int GROUP, bool BF16>
cudaError_t launch_t(const LatParams& p, const CUtensorMap& map, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  auto kern = latent_kernel<GROUP, BF16>;
  if (const cudaError_t e = allow_smem_once(kern, SMEM, &done); e != cudaSuccess) return e;
  return launch_chained(kern, dim3(grid), THREADS, SMEM, st, map, p);
}

}  // namespace

cudaError_t launch_latent_cache(const LatParams& p, const CUtensorMap& q, bool bf16, int group, int sms,
                                cudaStream_t st) {
  const int grid = imin(sms, kLatMaxCtas) / group * group;
  if (group == 1) return bf16 ? launch_t<1, true>(p, q, grid, st) : launch_t<1, false>(p, q, grid, st);
  return bf16 ? launch_t<2, true>(p, q, grid, st) : launch_t<2, false>(p, q, grid, st);
}

cudaError_t launch_latent_lists(const LatParams& p, const CUtensorMap& q, bool bf16, int sms, cudaStream_t st) {
  const int64_t units = static_cast<int64_t>(p.B) * p.S * p.HKV * p.splits;
  const int grid = static_cast<int>(units < sms ? units : sms);
  const cudaError_t e = bf16 ? launch_t<0, true>(p, q, grid, st) : launch_t<0, false>(p, q, grid, st);
  return e != cudaSuccess || p.splits == 1 ? e : launch_latent_join(p, bf16, 0, 0, sms, st);
}

}  // namespace ab
