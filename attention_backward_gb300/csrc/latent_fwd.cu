// The expanded form of latent attention for prompts (include/attn_latent.h): each
// head has keys of 128 columns of its own beside 64 rotated ones that all heads
// share, and values of 128,
//   S = Qn Kn_h^T + Qr Kr^T,  O = softmax(S) V_h,  LSE.
//
// The dense forward's structure (dense_fwd.cu): persistent CTAs, units of two
// 128-row query tiles of one head, two softmax warpgroups with a row a thread, S
// and P in tensor memory, O rescaled only when a row's max has grown by 2^8.  The
// shared keys are read where they lie, as the third 64-column slab of every head's K,
// so that no [S, H, 192] keys are ever written.
//
// The pairs of tiles of the last, unfinished round of CTAs (all, where they are few) split
// their key blocks over the CTAs; f32 partials go to the workspace, and a second launch
// joins them in order.
//
// Two Q tiles of 192 columns leave room for 8 slabs of 128 keys x 64 columns: K
// and V come through a ring of slabs (three of K_j, two of V_j, ...), so that the next
// K is there while V is in use.
//
// A packed sequence's last block may reach rows of the next one, or rows that belong
// to none: those rows of V are zeroed in shared memory before the slab is published
// (a zero P times a NaN would be NaN; of K they only make scores that are masked).
//
// Bound by the tensor core.  Whole calls with the join, back to back: 4096 queries on 4096
// keys, 64 heads, no mask 434 us, 1580 TFLOP/s, 83 % of the bf16 peak (up to 478 where the
// power cap holds the clock down); 2048 on 8192, causal 432 us, 1390, of which the join 10;
// four packed sequences of 16384 together, 16 heads 325 us, 1310 (units of few key blocks begin
// and end often); 1024 packed sequences of 16, 4 heads 130 us.  What the
// products wait for is the softmax of the other tile, 1400 cycles a block beside 1280 of
// products.  (One lane issues, and waits on as few barriers as there are: with waits and
// commits of the whole warp between P's products and the next scores the first of these took
// 490 us.)  Half of the softmax are the 128 powers, 600 cycles; without a max, which the
// weights' sum can stand for, the compiler has too few registers to overlap them (439 us), and
// twice the warps with half a row each share the powers' unit (463).
//
// Warp roles (12 warps): 0-3 softmax of tile 0, 4-7 of tile 1, 8 TMA producer, 9 and
// 10 MMA issue of a tile each, 11 idle.  Every wait is bounded.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#define AB_INLINE_WAITS 1
#include "common.cuh"
#include "cvt.cuh"
#include "kv_launch.h"
#include "latent.h"
#include "latent_issue.cuh"
#include "sm103.cuh"

namespace ab {

namespace {

constexpr int BQ = 128;  // query rows per tile
constexpr int BK = 128;  // keys per block
constexpr int THREADS = 12 * 32;
// launched at 168 registers a thread (12 warps), re-split per warpgroup: the
// two softmax warpgroups hold a row of 128 scores each; the control warpgroup
// keeps the unit walk and the barrier phases of the persistent loop
constexpr uint32_t REG_SOFT = 208, REG_CTL = 88;
static_assert(2 * REG_SOFT + REG_CTL == 3 * 168, "register split must equal the launch's registers");
// A row's reference is set so that its largest weight is 2^7, and kept until one would
// pass 2^15: fp16 weights keep their normal range down to 2^-21 of the largest.
constexpr float kTop = 7.f, kRescaleLog2 = 8.f;
// From here on, where its steps are 1/2 and more, a reference is not taken off the scaled
// scores but off the scores themselves.  (From 2^27 on its rounding would pass the room that fp16 leaves.)
constexpr float kFar = 0x1p22f;

constexpr int D = 128;                 // value columns
constexpr int KSLABS = 3, VSLABS = 2;  // 64-column slabs of a row of Q or K, and of V
constexpr int BSLABS = KSLABS + VSLABS;
constexpr int SLAB = BQ * 128;         // [128 rows x 64 cols] 16-bit, 128-byte swizzled
constexpr int QTILE = KSLABS * SLAB;
constexpr int RING = 8;
constexpr int OFF_Q = 0;  // two query tiles
constexpr int OFF_R = OFF_Q + 2 * QTILE;
constexpr int OFF_BAR = OFF_R + RING * SLAB;
constexpr int OFF_MISC = OFF_BAR + 40 * 8;
constexpr int OFF_UNITS = OFF_MISC + 64;
constexpr int SMEM = OFF_UNITS + 128;
static_assert(SMEM <= 227 * 1024, "shared memory budget");
constexpr uint32_t T_S0 = 0, T_S1 = 128, T_O0 = 256, T_O1 = 256 + D;

// Where slab i of the ring lies.
__device__ __forceinline__ uint32_t slab_at(uint32_t i) { return OFF_R + i % RING * SLAB; }

// Score ``top`` as a reference in log2 units, and log2 of the factor that takes weights from
// reference ``x`` to ``top``.
__device__ __forceinline__ float scaled(float top, float scale) { return fmaf(top, scale, -kTop); }
__device__ __forceinline__ float below(float x, float top, float scale) {
  const float m = scaled(top, scale);
  return fabsf(m) >= kFar ? (x - top) * scale : scaled(x, scale) - m;
}

enum FwdBar : int {
  Q_FULL = 0,
  Q_EMPTY,            // every S MMA of both tiles of the unit has completed: the Q tiles may be reloaded
  K_FULL0,                    // K of every other block
  V_FULL0 = K_FULL0 + 2,      // and V
  K_EMPTY0 = V_FULL0 + 2,     // both tiles' products of it have completed
  V_EMPTY0 = K_EMPTY0 + 2,
  S_FULL0 = V_EMPTY0 + 2,     // per tile
  P_READY0 = S_FULL0 + 2,     // per tile and half of the keys: 4 softmax warps stored P
  O_DONE0 = P_READY0 + 4,     // per tile: the unit's P V MMAs completed
  O_FREE0 = O_DONE0 + 2,      // per tile: 4 softmax warps read the unit's O rows
  UNIT_FULL0 = O_FREE0 + 2,   // 2 ring slots: the producer published a unit
  UNIT_EMPTY0 = UNIT_FULL0 + 2,  // 2 ring slots: the 2 issuing and the 8 softmax warps read it
  TURN0 = UNIT_EMPTY0 + 2,  // per tile: the other one has issued its scores
  TAIL = TURN0 + 2,
  DRAIN0,  // of the issuing warps
  NUM_FWD_BARS = DRAIN0 + 2
};
static_assert(NUM_FWD_BARS <= 40, "barrier storage");

// The unit a CTA owns: two query tiles of one query head, both in one
// sequence (a dense batch row or a packed sequence), and each tile's block
// range [lo, hi) of 128-key blocks.
struct FwdUnit {
  int valid, b, h, seq_start, qlen, klen, off, q0;
  int index;  // in the launch's order
  int lo[2], hi[2];  // lo == hi: the tile sees no key; q0 + 128 w >= qlen: the tile is absent
};

// Key blocks [lo, hi) that query rows [q0, q1) of a row of ``qlen`` queries and
// ``klen`` keys see (query i at key position i + off).
__device__ __forceinline__ void key_block_range(int q0, int qlen, int klen, int off, int causal, int* lo, int* hi) {
  *lo = *hi = 0;
  if (q0 >= qlen || klen <= 0) return;
  const int q1 = imin(q0 + BQ, qlen);
  int64_t ke = klen;
  if (causal) {
    const int64_t e = static_cast<int64_t>(q1) + off;  // last visible key + 1
    ke = e < klen ? e : klen;
  }
  if (ke <= 0) return;
  *hi = static_cast<int>((ke + BK - 1) / BK);
}

// A packed sequence, and the pairs of those before it.
struct FwdPlace {
  int n, before;
};

// Unit u of the launch, longest first under a causal mask (the last query
// tiles of a row see the most keys): dense rows go through the tile pairs
// from the last, each over all (batch, head) pairs; packed sequences one after
// another, each the same way over its heads.  The pairs from p.whole on are p.splits
// units each, of an even share of their key blocks.  All lanes of a warp call it; ``at``:
// where a unit of a smaller number was found, or the start.  (A walk from the start for
// every unit and role took 0.59 s for 40000 sequences of 3 tokens.)
__device__ __forceinline__ FwdUnit decode_unit(int u, const LatFwdParams& p, FwdPlace* at) {
  FwdUnit t{};
  t.valid = 0;
  if (u < 0) return t;  // the end-of-work marker
  t.index = u;
  // my slot of partial rows; offsets that do not ascend may name more pairs than there are
  const int slot = u - p.whole;
  if (slot >= kLatFwdMaxUnits) return t;
  const int parts = slot >= 0 ? p.splits : 1, part = slot >= 0 ? slot % p.splits : 0;
  u = slot >= 0 ? p.whole + slot / p.splits : u;
  int pair = 0;
  if (p.cu_seqlens == nullptr) {
    const int np = (p.S + 2 * BQ - 1) / (2 * BQ);
    const int bh = p.B * p.H;
    if (u >= np * bh) return t;
    pair = np - 1 - u / bh;
    t.b = (u % bh) / p.H;
    t.h = (u % bh) % p.H;
    t.seq_start = 0;
    t.qlen = p.S;
    t.klen = p.Sk;
    t.off = p.Sk - p.S;
  } else {
    const int lane = threadIdx.x & 31;
    for (;; at->n += 32) {  // 32 sequences at once, each ((len + 255) / 256) * H pairs
      if (at->n >= p.num_seqs) return t;
      const int n = at->n + lane;
      int a = 0, len = 0;
      if (n < p.num_seqs) {
        a = clamp_pos(p.cu_seqlens[n], p.S);
        const int e = clamp_pos(p.cu_seqlens[n + 1], p.S);
        len = e > a ? e - a : 0;
      }
      const int mine = (len + 2 * BQ - 1) / (2 * BQ) * p.H;
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, u - at->before < upto);
      if (past == 0) {
        at->before += __shfl_sync(0xffffffffu, upto, 31);
        continue;
      }
      const int src = __ffs(past) - 1;
      at->n += src;
      at->before += __shfl_sync(0xffffffffu, upto - mine, src);
      t.seq_start = __shfl_sync(0xffffffffu, a, src);
      t.qlen = t.klen = __shfl_sync(0xffffffffu, len, src);
      break;
    }
    const int rem = u - at->before;
    pair = (t.qlen + 2 * BQ - 1) / (2 * BQ) - 1 - rem / p.H;
    t.h = rem % p.H;
    t.b = 0;
    t.off = 0;
  }
  t.q0 = pair * 2 * BQ;
  for (int w = 0; w < 2; ++w)
    key_block_range(t.q0 + w * BQ, t.qlen, t.klen, t.off, p.causal, &t.lo[w], &t.hi[w]);
  if (p.splits > 1) {
    const int n = imax(t.hi[0], t.hi[1]);  // (no window: the blocks of both tiles begin at 0)
    const int a = static_cast<int>(static_cast<int64_t>(n) * part / parts);
    const int e = static_cast<int>(static_cast<int64_t>(n) * (part + 1) / parts);
    for (int w = 0; w < 2; ++w) {
      t.lo[w] = imax(t.lo[w], a), t.hi[w] = imin(t.hi[w], e);
      if (t.hi[w] <= t.lo[w]) t.lo[w] = t.hi[w] = 0;
    }
  }
  t.valid = 1;
  return t;
}

// The blocks [J0, J1) of a unit that some tile sees (J0 == J1: none).
struct UnitSpan {
  bool has[2];
  int J0, J1;
};

__device__ __forceinline__ UnitSpan unit_span(const FwdUnit& u) {
  UnitSpan s;
  s.J0 = 0x7fffffff;
  s.J1 = 0;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    s.has[w] = u.lo[w] < u.hi[w];
    if (s.has[w]) {
      s.J0 = imin(s.J0, u.lo[w]);
      s.J1 = imax(s.J1, u.hi[w]);
    }
  }
  if (s.J1 == 0) s.J0 = 0;
  return s;
}

// Persistent: each CTA's producer takes the unit of its number, then draws units, longest
// first, from a counter in the workspace header (cleared by the host before the launch,
// where there are more units than CTAs), decodes each from the place of the one before
// and publishes it to the other roles through a two-slot ring in shared memory; a draw
// past the last unit ends every role.  Barrier phases run on across units (K and V by a
// block counter, the S and P barriers of a tile by that tile's block counter), and two
// barriers hand the shared Q tiles (Q_EMPTY: every S MMA of the unit has completed) and a
// tile's O accumulator (O_FREE: its softmax warps have read O) to the next unit.
template <bool BF16>
__global__ void __launch_bounds__(THREADS, 1) latent_fwd_kernel(const __grid_constant__ LatFwdMaps maps,
                                                               const LatFwdParams p) {
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + OFF_MISC + 8);
  FwdUnit* const ring = reinterpret_cast<FwdUnit*>(sm + OFF_UNITS);
  static_assert(sizeof(FwdUnit) <= 64, "two units");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---------------------------------------------------------------- set-up, beside the end of the launch before
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    mbar_init(&bars[Q_FULL], 1);
    mbar_init(&bars[Q_EMPTY], 2);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bars[K_FULL0 + w], 1);
      mbar_init(&bars[V_FULL0 + w], 1);
      mbar_init(&bars[K_EMPTY0 + w], 2);
      mbar_init(&bars[V_EMPTY0 + w], 2);
      mbar_init(&bars[TURN0 + w], 1);
      mbar_init(&bars[S_FULL0 + w], 1);
      mbar_init(&bars[P_READY0 + 2 * w], 4);
      mbar_init(&bars[P_READY0 + 2 * w + 1], 4);
      mbar_init(&bars[O_DONE0 + w], 1);
      mbar_init(&bars[O_FREE0 + w], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[UNIT_FULL0 + i], 1);
      mbar_init(&bars[UNIT_EMPTY0 + i], 10);
      mbar_init(&bars[DRAIN0 + i], 1);
    }
    mbar_init(&bars[TAIL], 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // (the join's blocks, let in at once, wait beside the last parts and slow them: 256 queries
  // on 3000 keys, 160 heads 77 -> 80 us)
  grid_dependency_wait();
  const bool aligned = (smem_u32(sm) & 1023u) == 0;  // the swizzled tiles need an aligned base
  // (the call's error word, which a wait sets after a second at the earliest)
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.err = aligned ? kErrNone : kErrAlign;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (!aligned) {
    if (warp == 9) tmem_dealloc(tmem, 512);
    return;
  }
  const WaitCtx wc{abort_flag, p.err, p.timeout_ns};
  // a unit lasts as long as its keys do: waits for one to begin or to be taken have
  // a limit of their own (any wait that runs out ends the others too)
  const WaitCtx wu{abort_flag, p.err, 64 * p.timeout_ns};
  auto finish = [&]() {
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
    if (warp == 9) {
      __syncwarp();
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
  };

  // the uc-th unit of this CTA (consumers): waits for the producer's draw and
  // hands the slot back; invalid once the draws are exhausted
  auto next_unit = [&](uint32_t uc, bool* okp) -> FwdUnit {
    const uint32_t slot = uc & 1;
    FwdUnit u{};
    u.valid = 0;
    if (!(*okp = mbar_wait_warp(&bars[UNIT_FULL0 + slot], (uc >> 1) & 1, wu, kErrWaitTile))) return u;
    u = ring[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[UNIT_EMPTY0 + slot]);
    return u;
  };

  if (warp >= 8) {
    setmaxnreg_dec<REG_CTL>();
    if (warp == 8) {
      // ============================================================ producer
      int q_pend = -1, tail_pend = -1;
      uint32_t qc = 0, kc = 0, vc = 0, tail_ph = 0;  // blocks so far
      bool ok = true;
      FwdPlace at{0, 0};
      for (uint32_t uc = 0; ok; ++uc) {
        const uint32_t slot = uc & 1;
        if (uc >= 2 && !(ok = mbar_wait_warp(&bars[UNIT_EMPTY0 + slot], ((uc >> 1) - 1) & 1, wu, kErrWaitTile)))
          break;
        int t = 0;
        if (uc == 0) {
          t = blockIdx.x;
        } else {
          const int ctas = gridDim.x;
          if (lane == 0) t = p.units > ctas ? ctas + atomicAdd(p.unit_counter, 1) : -1;
          t = __shfl_sync(0xffffffffu, t, 0);
        }
        const FwdUnit u = decode_unit(t, p, &at);
        if (lane == 0) {
          ring[slot] = u;
          mbar_arrive(&bars[UNIT_FULL0 + slot]);
        }
        if (!u.valid) break;
        const UnitSpan sp = unit_span(u);
        if (sp.J1 <= sp.J0) continue;
        // the previous unit's S MMAs have read its Q tiles
        if (qc >= 1 && !(ok = mbar_wait_warp(&bars[Q_EMPTY], (qc - 1) & 1, wc, kErrWaitStageEmpty))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars[Q_FULL], (sp.has[0] + sp.has[1]) * QTILE);
          for (int w = 0; w < 2; ++w) {
            if (!sp.has[w]) continue;
#pragma unroll
            for (int s = 0; s < KSLABS; ++s)
              tma_load_4d(sm + OFF_Q + w * QTILE + s * SLAB, &maps.q, &bars[Q_FULL], s * 64, u.h,
                          u.seq_start + u.q0 + w * BQ, u.b);
          }
        }
        q_pend = qc & 1;
        ++qc;
        for (int j = sp.J0; j < sp.J1 && ok; ++j) {
          const int pos = u.seq_start + j * BK;
          // slabs 5 kc to 5 kc + 2, behind a slab of K and both of V of two blocks ago
          if (kc >= 2 && !(ok = mbar_wait_warp(&bars[V_EMPTY0 + (kc & 1)], ((kc >> 1) - 1) & 1, wc, kErrWaitStageEmpty))) break;
          if (lane == 0) {
            uint64_t* const bar = &bars[K_FULL0 + (kc & 1)];
            mbar_arrive_expect_tx(bar, KSLABS * SLAB);
#pragma unroll
            for (int s = 0; s < KSLABS; ++s)
              tma_load_4d(sm + slab_at(BSLABS * kc + s), s < KSLABS - 1 ? &maps.kn : &maps.kr, bar,
                          s < KSLABS - 1 ? s * 64 : 0, s < KSLABS - 1 ? u.h : 0, pos, u.b);
          }
          ++kc;
          // the two behind them, where two slabs of the last K were
          if (vc >= 1 && !(ok = mbar_wait_warp(&bars[K_EMPTY0 + ((vc - 1) & 1)], ((vc - 1) >> 1) & 1, wc, kErrWaitStageEmpty))) break;
          // rows of the block behind the sequence's end (a dense row's read zeros)
          const int r0 = imin(u.klen - j * BK, BK), r1 = p.cu_seqlens ? imin(p.S - pos, BK) : 0;
          const bool tail = r0 < r1;
          const uint32_t s0 = BSLABS * vc + KSLABS;
          if (lane == 0) {
            uint64_t* const bar = &bars[tail ? static_cast<uint32_t>(TAIL) : V_FULL0 + (vc & 1)];
            mbar_arrive_expect_tx(bar, VSLABS * SLAB);
#pragma unroll
            for (int s = 0; s < VSLABS; ++s) tma_load_4d(sm + slab_at(s0 + s), &maps.v, bar, s * 64, u.h, pos, u.b);
          }
          if (tail) {
            // loaded onto the producer's own barrier, the rows zeroed, then published
            tail_pend = tail_ph & 1;
            if (!(ok = mbar_wait_warp(&bars[TAIL], tail_ph & 1, wc, kErrWaitTail))) break;
            tail_pend = -1;
            ++tail_ph;
            for (int s = 0; s < VSLABS; ++s) zero_tile_rows(sm + slab_at(s0 + s), 1, SLAB, r0, r1, lane);
            if (lane == 0) mbar_arrive(&bars[V_FULL0 + (vc & 1)]);
          }
          ++vc;
        }
      }
      // loads still in flight land before the CTA exits: the last Q and the last blocks'
      if (lane == 0) {
        if (q_pend >= 0) mbar_drain(&bars[Q_FULL], q_pend);
        if (tail_pend >= 0) mbar_drain(&bars[TAIL], tail_pend);
        for (uint32_t i = kc > 2u ? kc - 2 : 0u; i < kc; ++i) mbar_drain(&bars[K_FULL0 + (i & 1)], (i >> 1) & 1);
        for (uint32_t i = vc > 2u ? vc - 2 : 0u; i < vc; ++i) mbar_drain(&bars[V_FULL0 + (i & 1)], (i >> 1) & 1);
      }
      __syncwarp();
    } else if (warp < 11) {
      // ============================================================ MMA issue of tile w
      // A warp a tile: neither waits on the other's softmax, and the tensor core takes
      // what is there.  (One warp for both, unrolled, spent 4700 cycles a block on issue.)
      const int w = warp - 9;
      constexpr uint32_t IDESC_S = idesc_f16(BF16, 128, BK, false, false);
      constexpr uint32_t IDESC_PV = idesc_f16(BF16, 128, D, false, true), IDESC_PV1 = idesc_f16(BF16, 128, 64, false, true);
      const uint64_t q_kmaj = sdesc_sw128(smem_u32(sm) + OFF_Q, 16, 1024) + sdesc_step(QTILE) * w;
      const uint64_t r_kmaj = sdesc_sw128(smem_u32(sm) + OFF_R, 16, 1024);
      const uint64_t r_mn = sdesc_sw128(smem_u32(sm) + OFF_R, SLAB, 1024);
      const uint32_t ts = tmem + T_S0 + (T_S1 - T_S0) * w, to = tmem + T_O0 + (T_O1 - T_O0) * w;
      // One lane does all of it: a wait or a commit of the whole warp takes 70 to 140 cycles.
      if (elect_lane()) {
        uint32_t qc = 0, bc = 0, npv = 0, oc = 0;  // units, blocks, blocks and units of my tile so far
        bool ok = true;
        auto wait_k = [&](uint32_t b) { return mbar_wait(&bars[K_FULL0 + (b & 1)], (b >> 1) & 1, wc, kErrWaitKV); };
        // Block b's turn of my tile at the scores: tile 0's, then tile 1's, each issued in one
        // go: one's softmax then runs while the other's products do.  (Side by side, both
        // tiles' S end at the same time, and both softmaxes run with the tensor core idle.)
        auto turn = [&](uint32_t b) {
          if (w == 0 && b == 0) return true;
          const uint32_t n = w ? b : b - 1;
          return mbar_wait(&bars[TURN0 + w], n & 1, wc, kErrWaitTile);
        };
        auto pass = [&]() {
          mbar_arrive(&bars[TURN0 + 1 - w]);
        };
        // S of block b, whose K is there
        auto scores = [&](uint32_t b) {
          tc_fence_after();
#pragma unroll 1
          for (int s = 0; s < KSLABS; ++s) {
            const uint64_t q = q_kmaj + sdesc_step(SLAB) * s, k = r_kmaj + sdesc_step(SLAB) * ((BSLABS * b + s) % RING);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_ss_e(ts, q + sdesc_step(kk * 32), k + sdesc_step(kk * 32), IDESC_S, s + kk > 0, 1u);
          }
          mma_commit_1(&bars[S_FULL0 + w]);
          pass();
          mma_commit_1(&bars[K_EMPTY0 + (b & 1)]);
        };
        // block b goes without my tile
        auto skip_k = [&](uint32_t b) -> bool {
          if (!wait_k(b) || !turn(b)) return false;
          pass();
          mbar_arrive(&bars[K_EMPTY0 + (b & 1)]);
          return true;
        };
        for (uint32_t uc = 0; ok; ++uc) {
          if (!(ok = mbar_wait(&bars[UNIT_FULL0 + (uc & 1)], (uc >> 1) & 1, wu, kErrWaitTile))) break;
          const FwdUnit u = ring[uc & 1];
          mbar_arrive(&bars[UNIT_EMPTY0 + (uc & 1)]);
          if (!u.valid) break;
          const UnitSpan sp = unit_span(u);
          if (sp.J1 <= sp.J0) continue;
          const int J0 = sp.J0, J1 = sp.J1, lo = w ? u.lo[1] : u.lo[0], hi = w ? u.hi[1] : u.hi[0];
          auto in = [&](int j) { return lo <= j && j < hi; };
          if (!(ok = mbar_wait(&bars[Q_FULL], qc & 1, wc, kErrWaitStageFull))) break;
          ++qc;
          if (in(J0)) {
            if (!(ok = wait_k(bc) && turn(bc))) break;
            scores(bc);
          } else if (!(ok = skip_k(bc))) {
            break;
          }
          // (every S MMA of the unit issued: Q may be loaded anew)
          if (J0 + 1 >= hi) mma_commit_1(&bars[Q_EMPTY]);
          for (int j = J0; j < J1; ++j, ++bc) {
            const bool more = j + 1 < J1 && in(j + 1);
            if (!(ok = mbar_wait(&bars[V_FULL0 + (bc & 1)], (bc >> 1) & 1, wc, kErrWaitKV))) break;
            if (in(j)) {
              // my O accumulator: the softmax warps have read the previous unit's O
              if (j == lo && oc >= 1 && !(ok = mbar_wait(&bars[O_FREE0 + w], (oc - 1) & 1, wu, kErrWaitDQEmpty))) break;
              const uint32_t s0 = (BSLABS * bc + KSLABS) % RING, s1 = (BSLABS * bc + KSLABS + 1) % RING;
              const uint32_t acc = j > lo;
#pragma unroll 1
              for (int hf = 0; hf < 2; ++hf) {
                if (!(ok = mbar_wait(&bars[P_READY0 + 2 * w + hf], npv & 1, wc, kErrWaitP))) break;
                tc_fence_after();
                if (s1 == s0 + 1) {  // side by side: products of 128 columns
                  const uint64_t b = r_mn + sdesc_step(SLAB) * s0 + sdesc_step(4 * 2048) * hf;
#pragma unroll
                  for (int kk = 0; kk < BK / 32; ++kk)
                    mma_ts_e(to, ts + 32 * hf + kk * 8, b + sdesc_step(kk * 2048), IDESC_PV, kk > 0 ? 1u : acc | hf, 1u);
                } else {
#pragma unroll 1
                  for (int kk = 0; kk < BK / 32; ++kk) {
                    const uint64_t at = sdesc_step(2048) * (4 * hf + kk);
                    const uint32_t more_o = kk > 0 ? 1u : acc | hf;
                    mma_ts_e(to, ts + 32 * hf + kk * 8, r_mn + sdesc_step(SLAB) * s0 + at, IDESC_PV1, more_o, 1u);
                    mma_ts_e(to + 64, ts + 32 * hf + kk * 8, r_mn + sdesc_step(SLAB) * s1 + at, IDESC_PV1, more_o, 1u);
                  }
                }
              }
              if (!ok) break;
              ++npv;
              mma_commit_1(&bars[V_EMPTY0 + (bc & 1)]);
              if (j + 1 >= hi) mma_commit_1(&bars[O_DONE0 + w]);
            } else {
              mbar_arrive(&bars[V_EMPTY0 + (bc & 1)]);
            }
            if (more) {
              if (!(ok = wait_k(bc + 1) && turn(bc + 1))) break;
              scores(bc + 1);
              if (j + 2 >= hi) mma_commit_1(&bars[Q_EMPTY]);
            } else if (j + 1 < J1 && !(ok = skip_k(bc + 1))) {
              break;
            }
          }
          if (!ok) break;
          oc += lo < hi ? 1u : 0u;
        }
        // every MMA issued by this warp completes before TMEM is released
        mma_commit_1(&bars[DRAIN0 + w]);
        mbar_drain(&bars[DRAIN0 + w], 0);
      }
      __syncwarp();
    }
    // warp 11: nothing to do
    finish();
    return;
  }

  setmaxnreg_inc<REG_SOFT>();
  // ============================================================ softmax of tile w (lane = query row)
  const int w = warp >> 2, quad = warp & 3;
  const int row = quad * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t tS = tmem + lane_off + (w ? T_S1 : T_S0);
  const uint32_t tO = tmem + lane_off + (w ? T_O1 : T_O0);
  uint32_t c = 0, oc = 0;  // blocks of this tile over all units so far, and units with any
  bool ok = true;
  for (uint32_t uc = 0; ok; ++uc) {
    const FwdUnit u = next_unit(uc, &ok);
    if (!ok || !u.valid) break;
    const int qt0 = u.q0 + w * BQ;  // first (sequence-local) query of the tile
    if (qt0 >= u.qlen) continue;    // the tile is past the end of its sequence
    const int lo_w = w ? u.lo[1] : u.lo[0], hi_w = w ? u.hi[1] : u.hi[0];
    const int q = qt0 + row;
    const uint32_t c0 = c;
    float top = -INFINITY, l = 0.f;  // top: the score that is the row's reference
    bool far = false;
    for (int j = lo_w; j < hi_w; ++j, ++c) {
      if (!(ok = mbar_wait_warp(&bars[S_FULL0 + w], c & 1, wc, kErrWaitS))) break;
      tc_fence_after();
      uint32_t sr[BK];
#pragma unroll
      for (int ch = 0; ch < BK / 32; ++ch) tmem_ld32(tS + ch * 32, sr + ch * 32);
      tmem_ld_wait();
      const int k0 = j * BK;
      // every key and query of the block in range and inside the mask
      const bool full_vis = k0 + BK <= u.klen && qt0 + BQ <= u.qlen && (!p.causal || qt0 + u.off >= k0 + BK - 1);
      // row max over four independent chains
      float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (full_vis) {
#pragma unroll
        for (int k = 0; k < BK; ++k) mx4[k & 3] = fmaxf(mx4[k & 3], __uint_as_float(sr[k]));
      } else {
        // keys k < k_hi of the block are visible to my query
        const int64_t d0 = static_cast<int64_t>(q) + u.off - k0;  // my key position relative to the block
        int64_t hi = u.klen - k0;
        if (p.causal) hi = hi < d0 + 1 ? hi : d0 + 1;
        if (q >= u.qlen) hi = 0;
        const int k_hi = static_cast<int>(hi < 0 ? 0 : (hi > BK ? BK : hi));
#pragma unroll
        for (int k = 0; k < BK; ++k) {
          const float s = k < k_hi ? __uint_as_float(sr[k]) : -INFINITY;
          sr[k] = __float_as_uint(s);
          mx4[k & 3] = fmaxf(mx4[k & 3], s);
        }
      }
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
      // a row whose max grew past the threshold is rescaled; a row that had no
      // visible key so far adopts the max (its O row and l are zero)
      const float was = top;
      const bool grown = (mx - top) * p.scale_log2 > kRescaleLog2;
      if (grown) top = mx;
      const float m = top == -INFINITY ? 0.f : scaled(top, p.scale_log2);
      if (__any_sync(0xffffffffu, grown || far)) {
        far = fabsf(m) >= kFar;
        const bool resc = grown && was != -INFINITY;
        if (__any_sync(0xffffffffu, resc)) {
          // (the tile's previous P V, issued before these scores, has completed as they have)
          const float f = resc ? ex2(below(was, top, p.scale_log2)) : 1.f;
          l *= f;
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t r[32];
            tmem_ld32(tO + ch * 32, r);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
            tmem_st16(tO + ch * 32, r);
            tmem_st16(tO + ch * 32 + 16, r + 16);
          }
        }
        if (__any_sync(0xffffffffu, far)) {
          const float off = far ? top : 0.f;
#pragma unroll
          for (int k = 0; k < BK; ++k) sr[k] = __float_as_uint(__uint_as_float(sr[k]) - off);
        }
      }
      // S * scale - m two keys per instruction (f32x2 FMA), the row sum in two
      // f32x2 accumulators
      const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = far ? make_float2(kTop, kTop) : make_float2(-m, -m);
      float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int ch = 0; ch < BK / 32; ++ch) {
        uint32_t pw[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = __ffma2_rn(
              make_float2(__uint_as_float(sr[ch * 32 + 2 * e]), __uint_as_float(sr[ch * 32 + 2 * e + 1])), sc2, nm2);
          const float2 pp = make_float2(ex2(x.x), ex2(x.y));
          sum2[e & 1] = __fadd2_rn(sum2[e & 1], pp);
          pw[e] = pack2<BF16>(pp.x, pp.y);
        }
        // P pairs of keys 32ch .. 32ch + 31 into S columns 16ch .. 16ch + 15 (the
        // scores of this row were all loaded above)
        tmem_st16(tS + ch * 16, pw);
        if (ch & 1) {  // a half of P: its products run while the other one is made
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[P_READY0 + 2 * w + (ch >> 1)]);
        }
      }
      l += (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
    }
    if (!ok) break;
    // ---- O = O_w / l and the natural-log LSE of the row
    const bool had = c > c0;  // the tile saw a key block in this unit
    if (had) {
      if (!(ok = mbar_wait_warp(&bars[O_DONE0 + w], oc & 1, wc, kErrWaitDQFull))) break;
      ++oc;
      tc_fence_after();
    }
    const bool live = q < u.qlen;
    const int64_t pos = u.seq_start + q;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t part_row = static_cast<int64_t>(u.index - p.whole) * 2 * BQ + w * BQ + row;  // of a part
    if (live) {
      if (u.index >= p.whole) {
        p.part_ml[part_row] = make_float2(top, l);
      } else {
        p.lse[u.b * p.sl_b + u.h * p.sl_h + pos * p.sl_s] =
            l == 0.f ? -INFINITY : (scaled(top, p.scale_log2) + log2f(l)) * 0.69314718055994531f;
      }
    }
    uint8_t* const out = p.o + 2 * (u.b * p.so_b + pos * p.so_s + u.h * p.so_h);
#pragma unroll 1
    for (int ch = 0; ch < D / 32; ++ch) {
      uint32_t r[32];
      if (had) {
        tmem_ld32(tO + ch * 32, r);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) r[e] = 0u;
      }
      if (live && u.index >= p.whole) {
        if (l != 0.f) {  // (a part that saw no key of the row says nothing)
          float4* const dst = reinterpret_cast<float4*>(p.part_o + part_row * D + ch * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]), __uint_as_float(r[4 * e + 2]),
                                 __uint_as_float(r[4 * e + 3]));
        }
      } else if (live) {
#pragma unroll
        for (int c8 = 0; c8 < 4; ++c8) {
          uint4 v;
          v.x = pack2<BF16>(__uint_as_float(r[c8 * 8 + 0]) * inv, __uint_as_float(r[c8 * 8 + 1]) * inv);
          v.y = pack2<BF16>(__uint_as_float(r[c8 * 8 + 2]) * inv, __uint_as_float(r[c8 * 8 + 3]) * inv);
          v.z = pack2<BF16>(__uint_as_float(r[c8 * 8 + 4]) * inv, __uint_as_float(r[c8 * 8 + 5]) * inv);
          v.w = pack2<BF16>(__uint_as_float(r[c8 * 8 + 6]) * inv, __uint_as_float(r[c8 * 8 + 7]) * inv);
          *reinterpret_cast<uint4*>(out + 2 * (ch * 32 + c8 * 8)) = v;
        }
      }
    }
    if (had) {
      // this unit's O rows are read: the next unit's first P V may overwrite them
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[O_FREE0 + w]);
    }
  }
  finish();
}

// Joins the parts of split units: a warp a row, 4 columns a lane, the parts in order.
constexpr int JOIN_WARPS = 8;
template <bool BF16>
__global__ void __launch_bounds__(JOIN_WARPS * 32) latent_fwd_join_kernel(const LatFwdParams p, int pairs) {  // of the split pairs
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31, w = blockIdx.x * JOIN_WARPS + (threadIdx.x >> 5), pair = w / (2 * BQ), row = w % (2 * BQ);
  if (pair >= pairs) return;
  FwdPlace at{0, 0};
  const FwdUnit u = decode_unit(p.whole + pair * p.splits, p, &at);
  const int q = u.q0 + row;
  if (!u.valid || q >= u.qlen) return;
  const int64_t first = static_cast<int64_t>(pair) * p.splits * 2 * BQ + row;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < p.splits; i0 += 32) {
    const int n = imin(32, p.splits - i0);
    float2 v = make_float2(0.f, 0.f);
    if (lane < n) v = p.part_ml[first + static_cast<int64_t>(i0 + lane) * 2 * BQ];
    float mx = v.y == 0.f ? -INFINITY : v.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mx = fmaxf(mx, m);
    const float f = v.y == 0.f ? 0.f : ex2(below(v.x, mx, p.scale_log2));
    const float g = m == -INFINITY ? 0.f : ex2(below(m, mx, p.scale_log2));
    m = mx;
    float sum = f * v.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * g + sum;
    acc.x *= g, acc.y *= g, acc.z *= g, acc.w *= g;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
      if (fi == 0.f) continue;
      const float4 x = reinterpret_cast<const float4*>(p.part_o + (first + static_cast<int64_t>(i0 + i) * 2 * BQ) * D)[lane];
      acc.x += fi * x.x, acc.y += fi * x.y, acc.z += fi * x.z, acc.w += fi * x.w;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t pos = u.seq_start + q;
  *reinterpret_cast<uint2*>(p.o + 2 * (u.b * p.so_b + pos * p.so_s + u.h * p.so_h + 4 * lane)) =
      make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
  if (lane == 0)
    p.lse[u.b * p.sl_b + u.h * p.sl_h + pos * p.sl_s] = l == 0.f ? -INFINITY : (scaled(m, p.scale_log2) + log2f(l)) * 0.69314718055994531f;
}

template <bool BF16>
cudaError_t launch_t(const LatFwdParams& p, const LatFwdMaps& m, int split_pairs, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  auto kern = latent_fwd_kernel<BF16>;
  if (const cudaError_t e = allow_smem_once(kern, SMEM, &done); e != cudaSuccess) return e;
  if (const cudaError_t e = launch_chained(kern, dim3(grid), THREADS, SMEM, st, m, p); e != cudaSuccess || split_pairs == 0) return e;
  return launch_chained(latent_fwd_join_kernel<BF16>, dim3(split_pairs * (2 * BQ / JOIN_WARPS)), JOIN_WARPS * 32, 0,
                        st, p, split_pairs);
}

}  // namespace

cudaError_t launch_latent_fwd(const LatFwdParams& p, const LatFwdMaps& m, bool bf16, int split_pairs, int grid,
                              cudaStream_t st) {
  return bf16 ? launch_t<true>(p, m, split_pairs, grid, st) : launch_t<false>(p, m, split_pairs, grid, st);
}

}  // namespace ab
