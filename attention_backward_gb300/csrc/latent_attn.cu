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
//   P^T  = 2^(S^T scale log2 e - m)     16 bits, in shared memory
//   O^T += C^T P^T        four M-tiles of 128 latent columns, N = 64, K = 64 keys
//
// so that a tile is read once from memory, serves as K (K-major) and as C^T
// (M-major), and 512 columns of O fit tensor memory beside the scores: rows as M
// would need all of it.  Few rows cost no more products than 64.
//
// Softmax: the scores arrive as fragments of 16 keys x 64 rows a warp (a thread: 2
// keys, 16 rows).  A row's reference m is kept until a weight would pass 2^15:
// one vote of the four warps a tile, and only then is the max taken, l scaled and O^T
// scaled in tensor memory.  m is set so that the largest weight is 2^7: fp16 weights
// keep their normal range down to 2^-21 of it and steps of 2^-31.  l is summed from the f32
// weights, a thread's share of the keys in registers until the unit ends.
//
// Cache: the line of kv_sched.cuh, cut evenly over the CTAs; a unit split over
// several leaves f32 partials that latent_join.cu joins.  Where requests have more
// than 64 rows two CTAs share a part, 64 rows each of units of 128, so that the second
// reads its keys from L2.  Lists: a unit a token and KV group, longest lists first.
//
// Rows of a page come as TMA boxes; listed rows by 16-byte asynchronous copies of four
// warps, a slab's swizzle written by address.  (TMA gathers of four rows took 37 ns each,
// 5.4 us a tile, four times what the products and the softmax of one take.)
//
// Keys that nobody sees: scores of rows that were not loaded are masked; their 16-key
// groups are left out of the O products, and rows behind the last key inside a group are
// zeroed by the softmax warps (0 * NaN is NaN).  Listed rows that are not visible are
// filled with zeros.
//
// Warp roles (12 warps): 0-3 softmax and output, 4-7 loads of Q (lists: of listed rows),
// 8 pages (lists: Q), 9 MMA issue, 10 the walk, a unit ahead of the others, 11 idle.
// Every wait is bounded.
#include <cmath>

#include "cvt.cuh"
#include "kv_launch.h"
#include "kv_sched.cuh"
#include "latent.h"
#include "sm103.cuh"

namespace ab {

namespace {

constexpr int NR = kLatRows, KT = kLatKeys;
constexpr int NSLAB = kLatRow / 64;
constexpr int SLAB = KT * 128;  // [64 rows x 64 columns] 16-bit, 128-byte swizzled
constexpr int TILE = NSLAB * SLAB;
constexpr int STAGES = 2;
constexpr int kWarps = 12, THREADS = kWarps * 32;
constexpr float kTop = 7.f, kMost = 15.f;  // log2 of a row's largest weight when its max is taken, and of the most it may grow to
constexpr float kNone = -1e30f;            // reference of a row that has seen no key

enum LatBar : int {
  Q_FULL = 0,                // 4 loading warps (lists: a copy)
  Q_EMPTY,                   // every S of the unit has completed
  KV_FULL0,                  // per stage (lists: 4 loading warps)
  KV_EMPTY0 = KV_FULL0 + STAGES,
  S_FULL0 = KV_EMPTY0 + STAGES,  // per score buffer
  P_READY = S_FULL0 + 2,     // 4 softmax warps
  O_DONE,                    // the tile's O products, and all before them
  O_FREE,                    // 4 softmax warps read the unit's O
  UNIT_FULL0,                // 2 slots
  UNIT_EMPTY0 = UNIT_FULL0 + 2,  // 10 warps
  DRAIN = UNIT_EMPTY0 + 2,
  NUM_BARS
};

// A unit, or the CTA's part of one: key tiles [j0, j1).
struct LatUnit {
  int valid;  // 0: no more, 1: work, 2: nothing to do
  int n;      // request, or batch row
  int a, nq, L, off;  // first token of q, queries, visible positions, key position of query 0 (lists: a = token)
  int row0, live;     // first row in the request (lists: first head), rows of this CTA
  int j0, j1;
  int slot;  // -1: the whole unit, else the slot of its partial rows
};

struct LatShared {
  float mx[4][NR];    // per softmax warp and row: a max, or a sum
  float f[NR];        // per row: a factor
  float ref[NR];
  int hi[NR];         // keys that a row sees
  LatUnit units[2];
  uint32_t bits[STAGES][4];  // of a stage's tile and 16-key group: its keys that are loaded and visible, if its mask leaves them
  uint64_t bars[NUM_BARS];
  int64_t work[kWarps];
  uint32_t tmem;
  int abort;
};

constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + TILE;
constexpr int OFF_P = OFF_K + STAGES * TILE;
constexpr int OFF_SH = OFF_P + KT * 128;
constexpr int SMEM = OFF_SH + static_cast<int>(sizeof(LatShared));
static_assert(SMEM <= 227 * 1024, "shared memory budget");

constexpr uint32_t T_S = 0, T_O = 128;  // score buffers at 0 and 64; O^T tile m at 128 + 64 m

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// 16 lanes x 64 columns of a warp's quarter as fragments: registers 4 j + (0, 1) are
// row lane / 4, columns 8 j + 2 (lane % 4) + (0, 1); 4 j + (2, 3) row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag64(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, uint32_t bytes) {  // the rest reads zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// The four softmax warps; true in all of them if it is in one.
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 2, 128;" ::: "memory"); }

// ---------------------------------------------------------------- the walk along the line (one warp)

template <int RT>
__device__ __forceinline__ int64_t lanes_work(const KvAttnParams& p, const KvReq& r) {
  int64_t w = 0;
  const int nt = kv_row_tiles<RT>(r);
  for (int rt = threadIdx.x & 31; rt < nt; rt += 32) w += kv_row_tile<RT, KT>(r, rt, p).n + kLatCost;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  return w;
}

// Work of the requests [n0, n1), all lanes together.  A lane takes a request whose
// rows are one tile; the others are taken by all lanes.
template <int RT>
__device__ __forceinline__ int64_t requests_work(const KvAttnParams& p, int n0, int n1) {
  const int lane = threadIdx.x & 31;
  int64_t w = 0;
  for (int b = n0; b < n1; b += 32) {
    KvReq mine{};
    if (b + lane < n1) mine = kv_request(b + lane, p);
    if (mine.R > 0 && mine.R <= RT) w += kv_row_tile<RT, KT>(mine, 0, p).n + kLatCost;
    for (uint32_t m = __ballot_sync(0xffffffffu, mine.R > RT); m != 0; m &= m - 1) {
      const KvReq r = kv_request(b + __ffs(m) - 1, p);
      const int64_t all = lanes_work<RT>(p, r);
      if (lane == 0) w += all;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  return w;
}

struct LatCursor {
  int n, rt, pos;
};

// Cursor of position x counted from request n0 (x lies on the line).
template <int RT>
__device__ __forceinline__ LatCursor walk_to(const KvAttnParams& p, int n0, int64_t x) {
  const int lane = threadIdx.x & 31;
  LatCursor c{n0, 0, 0};
  for (int b = n0; b < p.N; b += 32) {
    KvReq mine{};
    if (b + lane < p.N) mine = kv_request(b + lane, p);
    bool found = false;
    int64_t w = mine.R > 0 && mine.R <= RT ? kv_row_tile<RT, KT>(mine, 0, p).n + kLatCost : 0;
    for (uint32_t m = __ballot_sync(0xffffffffu, mine.R > RT); m != 0; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const int64_t all = lanes_work<RT>(p, kv_request(b + src, p));
      if (lane == src) w = all;
    }
    int64_t inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, x < inc);
    if (past != 0) {
      const int src = __ffs(past) - 1;
      x -= __shfl_sync(0xffffffffu, inc - w, src);
      c.n = b + src;
      found = true;
    } else {
      x -= __shfl_sync(0xffffffffu, inc, 31);
    }
    if (found) break;
  }
  const KvReq r = kv_request(c.n, p);
  const int nt = kv_row_tiles<RT>(r);
  for (int b = 0; b < nt; b += 32) {
    const int64_t w = b + lane < nt ? kv_row_tile<RT, KT>(r, b + lane, p).n + kLatCost : 0;
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
    c.rt = b + src;
    c.pos = static_cast<int>(x - __shfl_sync(0xffffffffu, inc - w, src));
    break;
  }
  return c;
}

// GROUP: CTAs that share a part of the line; 0: index lists.
template <int GROUP, bool BF16>
__global__ void __launch_bounds__(THREADS, 1)
    latent_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ LatParams lp) {
  constexpr bool LISTS = GROUP == 0;
  constexpr int RT = NR * (LISTS ? 1 : GROUP);
  const KvAttnParams& p = lp.a;
  extern __shared__ __align__(1024) uint8_t sm[];
  LatShared& sh = *reinterpret_cast<LatShared*>(sm + OFF_SH);
  uint64_t* const bars = sh.bars;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  grid_dependency_wait();
  grid_dependents_launch();
  volatile int* const abort_flag = &sh.abort;
  const WaitCtx wc{abort_flag, LISTS ? p.err : p.cta_err + blockIdx.x, p.timeout_ns};
  // a unit lasts as long as its keys do: waits for one to begin or to be taken
  // have a limit of their own (any wait that runs out ends the others too)
  const WaitCtx wu{abort_flag, wc.err, 64 * p.timeout_ns};
  const bool aligned = (smem_u32(sm) & 1023u) == 0;
  if (threadIdx.x == 0) {
    if (LISTS) {
      if (!aligned) atomicCAS(p.err, 0, kErrAlign);
    } else {
      *wc.err = aligned ? kErrNone : kErrAlign;
      p.desc[blockIdx.x] = make_int4(0, 0, 0, -1);
    }
    sh.abort = 0;
  }
  // ---------------------------------------------------------------- the CTA's part of the line
  int64_t total = 0, begin = 0, end = 0;
  int parts = 1, per = 0;
  const int part = LISTS ? 0 : blockIdx.x / imax(GROUP, 1), sub = LISTS ? 0 : blockIdx.x % imax(GROUP, 1);
  if constexpr (!LISTS) {
    per = (p.N + kWarps - 1) / kWarps;
    const int64_t w = requests_work<RT>(p, imin(p.N, warp * per), imin(p.N, (warp + 1) * per));
    if (lane == 0) sh.work[warp] = w;
  }
  __syncthreads();
  if (!aligned) return;
  if constexpr (!LISTS) {
#pragma unroll
    for (int i = 0; i < kWarps; ++i) total += sh.work[i];
    if (total == 0) return;
    const int64_t want = (total + kLatMinWork - 1) / kLatMinWork;
    const int most = gridDim.x / GROUP;
    parts = want < most ? static_cast<int>(want) : most;
    if (part >= parts) return;
    begin = kv_part_begin(total, part, parts), end = kv_part_begin(total, part + 1, parts);
  }

  // ---------------------------------------------------------------- set-up
  if (threadIdx.x == 0) {
    mbar_init(&bars[Q_FULL], LISTS ? 1 : 4);
    mbar_init(&bars[Q_EMPTY], 1);
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&bars[KV_FULL0 + i], LISTS ? 4 : 1);
      mbar_init(&bars[KV_EMPTY0 + i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[S_FULL0 + i], 1);
      mbar_init(&bars[UNIT_FULL0 + i], 1);
      mbar_init(&bars[UNIT_EMPTY0 + i], 10);
    }
    mbar_init(&bars[P_READY], 4);
    mbar_init(&bars[O_DONE], 1);
    mbar_init(&bars[O_FREE], 4);
    mbar_init(&bars[DRAIN], 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

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

  if (warp == 10) {
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
      const int64_t units = static_cast<int64_t>(lp.B) * lp.S * lp.HKV;
      const int bg_n = lp.B * lp.HKV;
      uint32_t uc = 0;
      for (int64_t i = blockIdx.x;; i += gridDim.x, ++uc) {
        LatUnit u{};
        u.valid = i < units;
        if (u.valid) {
          // later tokens' lists are longest as a rule
          const int bg = static_cast<int>(i % bg_n), t = lp.S - 1 - static_cast<int>(i / bg_n);
          u.n = bg / lp.HKV, u.a = t;
          const int g = bg % lp.HKV;
          u.row0 = g * lp.gh, u.live = lp.gh;
          const int* const il = lp.idx + u.n * lp.si_b + t * lp.si_s + g * lp.si_h;
          int last = -1;
#pragma unroll 8
          for (int s = lane; s < lp.topk; s += 32) {
            const int j = il[s];
            if (j >= 0 && j < lp.SKV) last = s;
          }
          last = __reduce_max_sync(0xffffffffu, last);
          u.j1 = last < 0 ? 0 : last / KT + 1;
          u.slot = -1;
        }
        if (!publish(uc, u) || !u.valid) break;
      }
    } else {
      int w0 = 0;
      int64_t x = begin;
      while (x >= sh.work[w0]) x -= sh.work[w0++];
      LatCursor cur = walk_to<RT>(p, w0 * per, x);
      KvReq rq = kv_request(cur.n, p);
      x = begin;
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
  } else if (warp == 8) {
    uint32_t kc = 0, qc = 0;
    bool ok = true;
    for (uint32_t uc = 0; ok; ++uc) {
      const LatUnit u = next_unit(uc, &ok);
      if (!ok || !u.valid) break;
      if (u.valid == 2 || u.j1 <= u.j0) continue;
      if constexpr (LISTS) {
        // ========================================================== Q: 64 heads of the token (those past its group are not used)
        if (qc >= 1 && !(ok = mbar_wait_warp(&bars[Q_EMPTY], (qc - 1) & 1, wc, kErrWaitStageEmpty))) break;
        if (lane == 0) mbar_arrive_expect_tx(&bars[Q_FULL], TILE);
        __syncwarp();
        if (lane < NSLAB)
          tma_load_4d(sm + OFF_Q + lane * SLAB, &map, &bars[Q_FULL], lane * 64, u.row0, u.a, u.n);
        ++qc;
      } else {
        // ========================================================== pages
        // Lanes 0-3 look up the pages of a tile's 16-key groups, a tile ahead; a copy
        // takes 64 columns of a page's tokens in the tile.
        const int* const table = p.table + static_cast<int64_t>(u.n) * p.table_stride;
        const int span = p.page_log2 >= 6 ? 4 : 1 << (p.page_log2 - 4);  // groups a copy
        auto look_up = [&](int j) {
          const int k = j * KT + 16 * lane;
          const int page = lane < 4 && j < u.j1 && k < u.L ? table[k >> p.page_log2] : -1;
          return page < p.num_blocks ? page : -1;
        };
        int next = look_up(u.j0);
        for (int j = u.j0; j < u.j1; ++j, ++kc) {
          const int st = kc % STAGES;
          const uint32_t n = kc / STAGES;
          const int page = next;
          const uint32_t held = __ballot_sync(0xffffffffu, page >= 0);
          if (n >= 1 && !(ok = mbar_wait_warp(&bars[KV_EMPTY0 + st], (n - 1) & 1, wc, kErrWaitStageEmpty))) break;
          if (lane < 4) sh.bits[st][lane] = page >= 0 ? 0xffffu : 0u;
          __syncwarp();
          if (lane == 0) {
            int copies = 0;
            for (int g = 0; g < 4; g += span) copies += held >> g & 1;
            if (copies) mbar_arrive_expect_tx(&bars[KV_FULL0 + st], copies * span * 16 * 128 * NSLAB);
            else mbar_arrive(&bars[KV_FULL0 + st]);
          }
          __syncwarp();
          for (int i = lane; i - lane < 4 / span * NSLAB; i += 32) {
            const int g = i / NSLAB * span, s = i % NSLAB;
            const int pg = __shfl_sync(0xffffffffu, page, g & 3);
            if (g < 4 && pg >= 0)
              tma_load_4d(sm + OFF_K + st * TILE + s * SLAB + g * 2048, &map, &bars[KV_FULL0 + st], s * 64,
                          (j * KT + 16 * g) & ((1 << p.page_log2) - 1), pg, 0);
          }
          next = look_up(j + 1);
        }
      }
    }
    // copies in flight land before the CTA exits
    if (lane == 0) {
      if (qc >= 1) mbar_drain(&bars[Q_FULL], (qc - 1) & 1);
      for (uint32_t i = kc > static_cast<uint32_t>(STAGES) ? kc - STAGES : 0u; i < kc; ++i)
        mbar_drain(&bars[KV_FULL0 + i % STAGES], (i / STAGES) & 1);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ============================================================ MMA issue
    constexpr uint32_t IDESC_S = idesc_f16(BF16, KT, NR, false, false);
    constexpr uint32_t IDESC_O = idesc_f16(BF16, 128, NR, true, true);
    const uint32_t sbase = smem_u32(sm);
    const uint64_t k_kmaj = sdesc_sw128(sbase + OFF_K, 16, 1024);
    const uint64_t q_kmaj = sdesc_sw128(sbase + OFF_Q, 16, 1024);
    const uint64_t c_mn = sdesc_sw128(sbase + OFF_K, SLAB, 1024);
    const uint64_t p_mn = sdesc_sw128(sbase + OFF_P, 0, 1024);
    uint32_t kc = 0, qc = 0, oc = 0;
    bool ok = true;
    auto issue_s = [&](uint32_t i) {
      tc_fence_after();
      const uint32_t d = tmem + T_S + 64 * (i & 1);
      const uint64_t a = k_kmaj + sdesc_step((i % STAGES) * TILE);
#pragma unroll
      for (int s = 0; s < NSLAB; ++s)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss_w(d, a + sdesc_step(s * SLAB + kk * 32), q_kmaj + sdesc_step(s * SLAB + kk * 32), IDESC_S, s > 0 || kk > 0);
      mma_commit_w(&bars[S_FULL0 + (i & 1)]);
    };
    for (uint32_t uc = 0; ok; ++uc) {
      const LatUnit u = next_unit(uc, &ok);
      if (!ok || !u.valid) break;
      if (u.valid == 2 || u.j1 <= u.j0) continue;
      if (!(ok = mbar_wait_warp(&bars[Q_FULL], qc & 1, wc, kErrWaitStageFull))) break;
      ++qc;
      bool early = false;  // this tile's scores have been issued already
      bool begun = false;  // O holds something of this unit
      for (int j = u.j0; j < u.j1; ++j, ++kc) {
        const bool next = j + 1 < u.j1;
        if (!early) {
          if (!(ok = mbar_wait_warp(&bars[KV_FULL0 + kc % STAGES], (kc / STAGES) & 1, wc, kErrWaitKV))) break;
          issue_s(kc);
          if (!next) mma_commit_w(&bars[Q_EMPTY]);
        }
        early = false;
        // while the softmax works: the next tile's scores, if its rows are there
        if (next) {
          for (int spin = 0; spin < 4096; ++spin) {
            if (__any_sync(0xffffffffu, mbar_test(&bars[P_READY], kc & 1))) break;
            if (__all_sync(0xffffffffu, mbar_test(&bars[KV_FULL0 + (kc + 1) % STAGES], ((kc + 1) / STAGES) & 1))) {
              issue_s(kc + 1);
              if (j + 2 >= u.j1) mma_commit_w(&bars[Q_EMPTY]);
              early = true;
              break;
            }
          }
        }
        if (!(ok = mbar_wait_warp(&bars[P_READY], kc & 1, wc, kErrWaitP))) break;
        if (j == u.j0 && oc >= 1 && !(ok = mbar_wait_warp(&bars[O_FREE], (oc - 1) & 1, wc, kErrWaitDQEmpty))) break;
        tc_fence_after();
        const uint64_t a = c_mn + sdesc_step((kc % STAGES) * TILE);
        bool loaded[4] = {true, true, true, true};  // 16-key groups
        if constexpr (!LISTS) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) loaded[kk] = sh.bits[kc % STAGES][kk] != 0u && j * KT + 16 * kk < u.L;
        }
        if (loaded[0] && loaded[1] && loaded[2] && loaded[3]) {
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss_w(tmem + T_O + 64 * m, a + sdesc_step(2 * m * SLAB + kk * 2048), p_mn + sdesc_step(kk * 2048), IDESC_O,
                       begun || kk > 0);
          begun = true;
        } else {
#pragma unroll 1
          for (int kk = 0; kk < 4; ++kk) {
            if (!loaded[kk]) continue;
#pragma unroll
            for (int m = 0; m < 4; ++m)
              mma_ss_w(tmem + T_O + 64 * m, a + sdesc_step(2 * m * SLAB + kk * 2048), p_mn + sdesc_step(kk * 2048), IDESC_O,
                       begun);
            begun = true;
          }
        }
        mma_commit_w(&bars[KV_EMPTY0 + kc % STAGES]);
        mma_commit_w(&bars[O_DONE]);
      }
      ++oc;
    }
    // every product issued by this warp completes before tensor memory is released
    mma_commit_w(&bars[DRAIN]);
    if (lane == 0) mbar_drain(&bars[DRAIN], 0);
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    const int tid = threadIdx.x - 128;
    uint32_t qc = 0, kc = 0;
    bool ok = true, flushed = false;  // the tile before has been published already
    for (uint32_t uc = 0; ok; ++uc) {
      const LatUnit u = next_unit(uc, &ok);
      if (!ok || !u.valid) break;
      if (u.valid == 2 || u.j1 <= u.j0) continue;
      constexpr int PIECES = kLatRow / 8;  // 16-byte pieces of a row
      if constexpr (LISTS) {
        // ========================================================== listed rows: 16 of a tile a warp
        // A tile's copies are in flight while the next one's are issued.
        const int w = warp - 4, g = u.row0 / lp.gh;
        const int* const list = lp.idx + u.n * lp.si_b + static_cast<int64_t>(u.a) * lp.si_s + g * lp.si_h;
        const int64_t base = static_cast<int64_t>(u.n) * lp.SKV;
        auto look_up = [&](int j) {
          const int k = j * KT + 16 * w + (lane & 15);
          const int i = j < u.j1 && k < lp.topk ? list[k] : -1;
          return i >= 0 && i < lp.SKV ? i : -1;
        };
        auto publish = [&](uint32_t i) {  // tile i's copies of this warp have landed
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[KV_FULL0 + i % STAGES]);
        };
        int next = look_up(u.j0);
        for (int j = u.j0; j < u.j1; ++j, ++kc) {
          const int st = kc % STAGES;
          const uint32_t n = kc / STAGES;
          const int row = next;
          next = look_up(j + 1);
          const uint32_t seen = __ballot_sync(0xffffffffu, row >= 0) & 0xffffu;
          if (n >= 1 && j > u.j0 && !__all_sync(0xffffffffu, mbar_test(&bars[KV_EMPTY0 + st], (n - 1) & 1))) {
            // nothing to issue yet: the tile in flight is published meanwhile
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            publish(kc - 1);
            flushed = true;
          }
          ok = n < 1 || mbar_wait_warp(&bars[KV_EMPTY0 + st], (n - 1) & 1, wc, kErrWaitStageEmpty);
          if (!ok) break;
          if (lane == 0) sh.bits[st][w] = seen;
          uint8_t* const tile = sm + OFF_K + st * TILE;
#pragma unroll
          for (int r4 = 0; r4 < 16; r4 += 4) {
#pragma unroll
            for (int k = 0; k < 4 * PIECES / 32; ++k) {
              const int i = k * 32 + lane, r = r4 + i / PIECES, c = i % PIECES;
              const int at = __shfl_sync(0xffffffffu, row, r);
              const uint8_t* const src = lp.rows + (at < 0 ? 0 : 2 * (((base + at) * lp.HKV + g) * lp.row_stride + 8 * c));
              copy16_async(smem_u32(tile + (c >> 3) * SLAB + sw128_offset(16 * w + r, c & 7)), src, at < 0 ? 0 : 16);
            }
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (j > u.j0 && !flushed) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            publish(kc - 1);
          }
          flushed = false;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (ok && !flushed) publish(kc - 1);
        flushed = false;
      } else {
        // ========================================================== Q
        if (qc >= 1 && !(ok = mbar_wait_warp(&bars[Q_EMPTY], (qc - 1) & 1, wc, kErrWaitStageEmpty))) break;
        ++qc;
#pragma unroll 4
        for (int i = tid; i < NR * PIECES; i += 128) {
          const int r = i / PIECES, c = i % PIECES;
          const bool on = r < u.live;
          const int row = u.row0 + r;
          const uint8_t* src = p.q;
          if (on) src += 2 * (static_cast<int64_t>(u.a + row / p.G) * p.sq_s + (row % p.G) * p.sq_h + 8 * c);
          copy16_async(smem_u32(sm + OFF_Q + (c >> 3) * SLAB + sw128_offset(r, c & 7)), src, on ? 16 : 0);
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Q_FULL]);
      }
    }
  } else if (warp < 4) {
    // ============================================================ softmax and output
    const int tid = threadIdx.x;
    const int ka = 16 * warp + (lane >> 2), c0 = 2 * (lane & 3);  // my keys: ka, ka + 8; my rows: 8 j + c0 + (0, 1)
    const uint32_t quarter = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t bit_a = 1u << (ka & 15), bit_b = bit_a << 8;  // of group ``warp``
    uint32_t kc = 0;
    // The four warps meet at named barriers, which have no limit: a warp whose wait ran
    // out goes on (its results are void) to the next vote, where all four leave.
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
        if (tid < NR) kv_row_keys(r, (u.row0 + imin(tid, u.live - 1)) / p.G, p.causal, 0, &lo, &sh.hi[tid]);
        kv_row_keys(r, u.row0 / p.G, p.causal, 0, &lo, &hi_all);
        softmax_sync();
      }
      float ref[16], l[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) ref[c] = kNone, l[c] = 0.f;
      for (int j = u.j0; j < u.j1; ++j, ++kc) {
        const int st = kc % STAGES;
        wait(KV_FULL0 + st, (kc / STAGES) & 1, kErrWaitKV);  // (for its bits)
        const uint32_t b0 = sh.bits[st][0], b1 = sh.bits[st][1], b2 = sh.bits[st][2], b3 = sh.bits[st][3];
        wait(S_FULL0 + (kc & 1), (kc >> 1) & 1, kErrWaitS);
        tc_fence_after();
        uint32_t sr[32];
        tmem_ld_frag64(tmem + quarter + T_S + 64 * (kc & 1), sr);
        tmem_ld_wait();
        float* const s = reinterpret_cast<float*>(sr);
        if ((b0 & b1 & b2 & b3) != 0xffffu || (j + 1) * KT > hi_all) {
          const uint32_t w = sh.bits[st][warp];
          const bool va = w & bit_a, vb = w & bit_b;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int h = LISTS ? 0x7fffffff : sh.hi[8 * (c >> 1) + c0 + (c & 1)];
            float& x = s[4 * (c >> 1) + (c & 1)];
            float& y = s[4 * (c >> 1) + 2 + (c & 1)];
            if (!va || j * KT + ka >= h) x = -INFINITY;
            if (!vb || j * KT + ka + 8 >= h) y = -INFINITY;
          }
        }
        float over = -INFINITY;  // log2 of my largest weight
#pragma unroll
        for (int c = 0; c < 16; ++c)
          over = fmaxf(over, fmaf(fmaxf(s[4 * (c >> 1) + (c & 1)], s[4 * (c >> 1) + 2 + (c & 1)]), p.scale_log2, -ref[c]));
        if (softmax_any(over > kMost || bad)) {
          // ---- some row's weights outgrow the type: new references for those
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float m = fmaxf(s[4 * (c >> 1) + (c & 1)], s[4 * (c >> 1) + 2 + (c & 1)]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane < 4) sh.mx[warp][8 * (c >> 1) + c0 + (c & 1)] = m;
          }
          if ((dead = softmax_any(bad))) break;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int row = 8 * (c >> 1) + c0 + (c & 1);
            const float m = fmaxf(fmaxf(sh.mx[0][row], sh.mx[1][row]), fmaxf(sh.mx[2][row], sh.mx[3][row])) * p.scale_log2;
            float f = 1.f;
            if (m - ref[c] > kMost) {
              f = ref[c] == kNone ? 0.f : ex2(ref[c] - (m - kTop));
              ref[c] = m - kTop;
            }
            l[c] *= f;
            if (warp == 0 && lane < 4) sh.f[row] = f;
          }
          softmax_sync();
          if (j > u.j0) {
            // O^T of the tiles so far, once their products have completed
            wait(O_DONE, (kc - 1) & 1, kErrWaitDQFull);
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < 8; ++h) {
              const uint32_t at = tmem + quarter + T_O + 32 * h;
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
        if (!LISTS && (u.L & 15) && j == (u.L - 1) / KT) {
          // rows behind the last key of its group: the scores have been made, the O products follow
          const int r0 = u.L & (KT - 1), n = (16 - (u.L & 15)) * 64;
          for (int i = tid; i < n; i += 128)
            *reinterpret_cast<uint4*>(sm + OFF_K + st * TILE + (i & 7) * SLAB + (r0 + (i >> 6)) * 128 + (i >> 3 & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        uint32_t pa[8], pb[8];
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          const float x0 = ex2(fmaf(s[2 * c], p.scale_log2, -ref[c])), x1 = ex2(fmaf(s[2 * c + 1], p.scale_log2, -ref[c + 1]));
          const float y0 = ex2(fmaf(s[2 * c + 2], p.scale_log2, -ref[c])), y1 = ex2(fmaf(s[2 * c + 3], p.scale_log2, -ref[c + 1]));
          l[c] += x0 + y0, l[c + 1] += x1 + y1;
          pa[c / 2] = pack2<BF16>(x0, x1), pb[c / 2] = pack2<BF16>(y0, y1);
        }
        // the previous tile's O products have read P
        if (kc >= 1) wait(O_DONE, (kc - 1) & 1, kErrWaitDSFree);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          *reinterpret_cast<uint32_t*>(sm + OFF_P + sw128_offset(ka, c) + 2 * c0) = pa[c];
          *reinterpret_cast<uint32_t*>(sm + OFF_P + sw128_offset(ka + 8, c) + 2 * c0) = pb[c];
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[P_READY]);
      }
      if (dead) break;
      // ---- the rows' sums, then O
      const bool had = u.j1 > u.j0;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], o);
        if (lane < 4) {
          const int row = 8 * (c >> 1) + c0 + (c & 1);
          sh.mx[warp][row] = l[c];
          if (warp == 0) sh.ref[row] = ref[c];
        }
      }
      softmax_sync();
      // a row's place in o (lists: heads of a token; else query and head of the request)
      auto o_at = [&](int r) -> int64_t {
        if constexpr (LISTS) return u.n * lp.so_b + u.a * p.so_s + (u.row0 + r) * p.so_h;
        const int row = u.row0 + r;
        return static_cast<int64_t>(u.a + row / p.G) * p.so_s + (row % p.G) * p.so_h;
      };
      if (tid < NR) {
        const float sum = (sh.mx[0][tid] + sh.mx[1][tid]) + (sh.mx[2][tid] + sh.mx[3][tid]);
        sh.f[tid] = sum == 0.f ? 0.f : 1.f / sum;
        if (tid < u.live) {
          if (u.slot < 0) {
            const float lse = sum == 0.f ? -INFINITY : (sh.ref[tid] + log2f(sum)) * 0.69314718055994531f;
            if constexpr (LISTS) {
              p.lse[u.n * lp.sl_b + (u.row0 + tid) * p.sl_h + u.a * p.sl_s] = lse;
            } else {
              const int row = u.row0 + tid;
              p.lse[(row % p.G) * p.sl_h + static_cast<int64_t>(u.a + row / p.G) * p.sl_s] = lse;
            }
          } else {
            p.part_ml[static_cast<int64_t>(u.slot) * NR + tid] = make_float2(sh.ref[tid], sum);
          }
        }
      }
      softmax_sync();
      if (had) {
        wait(O_DONE, (kc - 1) & 1, kErrWaitDQFull);
        tc_fence_after();
      }
#pragma unroll 1
      for (int h = 0; h < 8; ++h) {
        const int d = 128 * (h >> 1) + tid, r0 = 32 * (h & 1);  // my latent column, first row
        if (r0 >= u.live) continue;
        uint32_t r[32];
        if (had) {
          tmem_ld32(tmem + quarter + T_O + 32 * h, r);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = 0u;
        }
        if (u.slot >= 0) {
          float* const out = p.part_o + (static_cast<int64_t>(u.slot) * NR + r0) * kLatDim + d;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (r0 + e < u.live) out[e * kLatDim] = __uint_as_float(r[e]);
        } else {
          // neighbouring lanes swap, so that each stores two columns of one row of a pair
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            // (a row that has seen no key may find anything in O)
            const float f0 = sh.f[r0 + e], f1 = sh.f[r0 + e + 1];
            const float x = f0 == 0.f ? 0.f : __uint_as_float(r[e]) * f0, y = f1 == 0.f ? 0.f : __uint_as_float(r[e + 1]) * f1;
            const float z = __shfl_xor_sync(0xffffffffu, lane & 1 ? x : y, 1);
            const uint32_t w = lane & 1 ? pack2<BF16>(z, y) : pack2<BF16>(x, z);
            const int row = r0 + e + (lane & 1);
            if (row < u.live) *reinterpret_cast<uint32_t*>(p.o + 2 * (o_at(row) + (d & ~1))) = w;
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
  if (warp == 9) {
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

cudaError_t launch_latent_cache(const LatParams& p, const CUtensorMap& pages, bool bf16, int group, int sms,
                                cudaStream_t st) {
  const int grid = imin(sms, kLatMaxCtas) / group * group;
  if (group == 1) return bf16 ? launch_t<1, true>(p, pages, grid, st) : launch_t<1, false>(p, pages, grid, st);
  return bf16 ? launch_t<2, true>(p, pages, grid, st) : launch_t<2, false>(p, pages, grid, st);
}

cudaError_t launch_latent_lists(const LatParams& p, const CUtensorMap& q, bool bf16, int sms, cudaStream_t st) {
  const int64_t units = static_cast<int64_t>(p.B) * p.S * p.HKV;
  const int grid = static_cast<int>(units < sms ? units : sms);
  return bf16 ? launch_t<0, true>(p, q, grid, st) : launch_t<0, false>(p, q, grid, st);
}

}  // namespace ab
