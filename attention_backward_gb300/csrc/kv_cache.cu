// Block tables and slot maps from request lengths, and the quantising write of
// new keys and values into the paged 8-bit cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "cvt.cuh"
#include "kv_cache.h"
#include "kv_launch.h"
#include "sm103.cuh"

namespace ab {

namespace {

// ---------------------------------------------------------------- tables

constexpr int kTabThreads = 512;

struct Need {
  int64_t tokens, pages;  // new tokens, pages inside the table's width
  int64_t wide;           // pages past the table's width
};

__device__ __forceinline__ Need request_need(int n, const KvTablesParams& p, int64_t* ctx_out, int64_t* before_out) {
  const int64_t ctx = imax(p.ctx[n], 0), add = imax(p.add[n], 0);
  const int64_t P1 = (int64_t(1) << p.page_log2) - 1;
  const int64_t before = (ctx + P1) >> p.page_log2, after = (ctx + add + P1) >> p.page_log2;
  const int64_t b = before < p.max_blocks ? before : p.max_blocks, a = after < p.max_blocks ? after : p.max_blocks;
  *ctx_out = ctx;
  *before_out = before;
  Need d;
  d.tokens = add;
  d.pages = a - b;
  d.wide = (after - before) - d.pages;
  return d;
}

// One launch, latency-bound (lengths in, 8 bytes a token out).  Every block
// repeats the scan over the requests (a thread sums ceil(N / 512) consecutive
// ones, then a block scan), which is cheaper than a second launch or a wait
// between blocks: 256 requests are one load a thread.  Each block then writes
// its share of the requests (a warp per request) and of the tokens (a search
// over the 512 sums in shared memory, then a walk inside one thread's
// requests).  Slots of fresh pages are computed from the free list, not read
// back from the table, so blocks do not depend on one another.  3.7 us for 256
// requests of one token, 4.5 us for 97 requests of 100753 tokens together.  A token's
// request is found by a walk inside a thread's share of them, ceil(N / 512), for each
// token: made for thousands of requests, its work grows with N^2 (one token each,
// whole calls: 27 us, the host's, up to 4096 requests, 72 us for 16384, 0.38 ms for
// 65536, 45 ms for 2^20).
__global__ void __launch_bounds__(kTabThreads) kv_tables_kernel(const KvTablesParams p) {
  __shared__ int64_t s_tok[kTabThreads + 1], s_pg[kTabThreads + 1];
  __shared__ int64_t w_tok[kTabThreads / 32], w_pg[kTabThreads / 32], w_wide[kTabThreads / 32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = (p.N + kTabThreads - 1) / kTabThreads;
  const int64_t start = p.free_start ? imax(*p.free_start, 0) : 0;
  const int64_t avail = p.num_free > start ? p.num_free - start : 0;
  Need sum{0, 0, 0};
  for (int i = 0; i < K; ++i) {
    const int64_t n = static_cast<int64_t>(tid) * K + i;
    if (n >= p.N) break;
    int64_t c, b;
    const Need d = request_need(static_cast<int>(n), p, &c, &b);
    sum.tokens += d.tokens, sum.pages += d.pages, sum.wide += d.wide;
  }
  int64_t it = sum.tokens, ip = sum.pages, iw = sum.wide;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, it, o), b = __shfl_up_sync(0xffffffffu, ip, o),
                  c = __shfl_up_sync(0xffffffffu, iw, o);
    if (lane >= o) it += a, ip += b, iw += c;
  }
  if (lane == 31) w_tok[warp] = it, w_pg[warp] = ip, w_wide[warp] = iw;
  __syncthreads();
  int64_t bt = 0, bp = 0, wide = 0;
  for (int w = 0; w < kTabThreads / 32; ++w) {
    if (w < warp) bt += w_tok[w], bp += w_pg[w];
    wide += w_wide[w];
  }
  s_tok[tid] = bt + it - sum.tokens;
  s_pg[tid] = bp + ip - sum.pages;
  if (tid == kTabThreads - 1) s_tok[kTabThreads] = bt + it, s_pg[kTabThreads] = bp + ip;
  __syncthreads();
  const int64_t tokens = s_tok[kTabThreads], pages = s_pg[kTabThreads];
  auto free_page = [&](int64_t i) -> int {  // the i-th page of this call
    if (i >= avail) return -1;
    const int b = p.free_blocks[start + i];
    return b >= 0 && b < p.num_blocks ? b : -1;
  };
  // what the requests before n of its thread's share need
  auto prefix = [&](int n, int64_t* tok, int64_t* pg) {
    const int o = n / K;
    *tok = s_tok[o], *pg = s_pg[o];
    for (int m = o * K; m < n; ++m) {
      int64_t c, b;
      const Need d = request_need(m, p, &c, &b);
      *tok += d.tokens, *pg += d.pages;
    }
  };
  if (blockIdx.x == 0 && tid == 0) {
    const int64_t taken = pages < avail ? pages : avail;
    int64_t lacking = wide + (pages - taken) + (tokens > p.T ? tokens - p.T : 0);
    lacking = lacking < 0x7fffffff ? lacking : 0x7fffffff;
    p.counts[0] = static_cast<int>(tokens < 0x7fffffff ? tokens : 0x7fffffff);
    p.counts[1] = static_cast<int>(taken);
    p.counts[2] = static_cast<int>(lacking);
    p.cu[0] = 0;
  }
  const int warps = gridDim.x * (kTabThreads / 32);
  for (int n = blockIdx.x * (kTabThreads / 32) + warp; n < p.N; n += warps) {
    int64_t tok, pg, ctx, before;
    prefix(n, &tok, &pg);
    const Need d = request_need(n, p, &ctx, &before);
    if (lane == 0) {
      const int64_t e = tok + d.tokens, len = ctx + d.tokens;
      p.cu[n + 1] = static_cast<int>(e < p.T ? e : p.T);
      p.kv_lens[n] = static_cast<int>(len < 0x7fffffff ? len : 0x7fffffff);
    }
    int* row = p.table + n * p.table_stride;
    for (int64_t j = lane; j < d.pages; j += 32) row[before + j] = free_page(pg + j);
  }
  const int threads = gridDim.x * kTabThreads;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTabThreads + tid; t < p.T; t += threads) {
    int slot = -1;
    int64_t pos = 0;
    if (t < tokens) {
      int lo = 0, hi = kTabThreads;  // the thread whose requests hold token t: s_tok[lo] <= t < s_tok[lo + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tok[mid] <= t) lo = mid;
        else hi = mid;
      }
      int64_t tok = s_tok[lo], pg = s_pg[lo], ctx = 0, before = 0;
      int n = lo * K;
      while (true) {
        const Need d = request_need(n, p, &ctx, &before);
        if (t < tok + d.tokens) break;
        tok += d.tokens, pg += d.pages;
        ++n;
      }
      pos = ctx + t - tok;
      const int64_t page = pos >> p.page_log2;
      if (page < p.max_blocks) {
        const int b = page < before ? p.table[n * p.table_stride + page] : free_page(pg + page - before);
        if (b >= 0 && b < p.num_blocks)
          slot = (b << p.page_log2) + static_cast<int>(pos & ((int64_t(1) << p.page_log2) - 1));
      }
    }
    p.slot_map[t] = slot;
    p.positions[t] = static_cast<int>(pos);
  }
}

// ---------------------------------------------------------------- write

constexpr int kWrThreads = 256;
constexpr int kWrGap = 32;  // tokens of a run are at most this far apart

// Two bytes of e4m3 to f32, and back (nearest, ties to even, +-448 beyond).
__device__ __forceinline__ float2 from_e4m3x2(uint32_t b) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(b), __NV_E4M3);
  return __half22float2(__half2(h));
}
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Least power of two s >= 2^-100 with amax <= 448 s (448 = 1.75 * 2^8).
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased; subnormals land below
  e = e < 27 ? 27 : e;
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// A team of W = page / 16 warps per (run, head, tensor): a warp holds 16 tokens
// of the run in registers (two 16-byte loads in flight a lane and token pair, all
// at once), the team joins their largest value in shared memory, and the bytes
// are written from the registers, so that x is read once.  (One warp a run, with
// a second read from L2, took 38.6 us on 33771 tokens of 4 heads of 128 in pages
// of 64, latency-bound.)  A block takes a window of TW tokens and as many of the
// 2 HKV (tensor, head) rows as it has teams; one ballot over the window's slots
// finds the runs that start in it, and its teams share them.  TW grows with the
// tokens: a window without a run's start is a block for nothing, one with many
// keeps them waiting.  A run with skipped tokens inside, or a page's scale that is
// no power of two, takes a second read (and true divisions) instead.
// Bound by its chain of loads (slots, values, the page's scale) at four blocks an
// SM: 23 us, 4.5 TB/s, on the 33771 tokens above; 5.4 us for 256 single tokens of 8
// heads of 128.
template <int D, bool BF16, int W>
__global__ void __launch_bounds__(kWrThreads, 4) kv_write_kernel(const KvWriteParams p, int TW) {
  constexpr int TEAMS = kWrThreads / 32 / W;
  constexpr int LPT = D / 8;      // lanes per token: 8 values (16 bytes) a lane
  constexpr int TPW = 32 / LPT;   // tokens per warp load
  constexpr int LOADS = 16 / TPW;
  __shared__ float s_max[2][kWrThreads / 32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / W, tw = warp % W;
  const int P = 1 << p.page_log2;
  const int64_t slots = static_cast<int64_t>(p.num_blocks) << p.page_log2;
  const int t0 = blockIdx.x * TW;
  const int t = t0 + lane;
  auto valid = [&](int s) { return s >= 0 && s < slots; };
  bool begins = false;
  const int my_slot = lane < TW && t < p.T ? p.slot_map[t] : -1;
  if (lane < TW && t < p.T) {
    const int s = my_slot;
    if (valid(s)) {
      // the valid token before mine, at most kWrGap tokens back
      int before = -1;
#pragma unroll 1
      for (int k = 1; k <= kWrGap && k <= t; ++k) {
        before = p.slot_map[t - k];
        if (valid(before)) break;
        before = -1;
      }
      begins = before < 0 || (before >> p.page_log2) != (s >> p.page_log2) || before >= s;
    }
  }
  const uint32_t runs = __ballot_sync(0xffffffffu, begins);
  const int nruns = __popc(runs);
  const int row0 = blockIdx.y * TEAMS, rows = imin(TEAMS, 2 * p.HKV - row0);
  int buf = 0;
  for (int item = team; item < nruns * rows; item += TEAMS, buf ^= 1) {
    uint32_t rest = runs;
    for (int i = item / rows; i > 0; --i) rest &= rest - 1;
    const int row = row0 + item % rows;
    const int which = row >= p.HKV ? 1 : 0, h = row - which * p.HKV;
    const int ts = t0 + __ffs(rest) - 1;
    const int slot = __shfl_sync(0xffffffffu, my_slot, __ffs(rest) - 1);
    const int blk = slot >> p.page_log2, off = slot & (P - 1);
    // Tokens [ts, ts + len): up to the first valid one that begins a run itself.
    // First the tokens in consecutive slots, all looked up at once; the loop then
    // looks whether others of the page follow.
    int len = 1;
    {
      const int most = imin(P - off, p.T - ts);
      int ahead[W == 1 ? 1 : W / 2];
#pragma unroll
      for (int k = 0; k < (W == 1 ? 1 : W / 2); ++k) {
        const int i = 1 + 32 * k + lane;
        ahead[k] = i < most ? p.slot_map[ts + i] - i : -1;
      }
      bool on = true;
#pragma unroll
      for (int k = 0; k < (W == 1 ? 1 : W / 2); ++k) {
        const uint32_t other = __ballot_sync(0xffffffffu, ahead[k] != slot);
        if (on) len += other ? __ffs(other) - 1 : 32;
        on = on && other == 0;
      }
      len = imin(len, most);
    }
    int last = slot + len - 1, count = len;  // last: slot of the valid token at ts + len - 1; count: valid ones
#pragma unroll 1
    while ((last & (P - 1)) != P - 1) {
      const int base = ts + len;  // 32 tokens from here on
      const int s = base + lane < p.T ? p.slot_map[base + lane] : -1;
      const uint32_t v = __ballot_sync(0xffffffffu, valid(s));
      if (v == 0) break;  // (kWrGap = 32: nothing later belongs to the run)
      const uint32_t below = v & ((1u << lane) - 1u);
      const int from = below ? 31 - __clz(below) : 0;
      const int sb = __shfl_sync(0xffffffffu, s, from);
      const int before = below ? sb : last;
      const bool ends = valid(s) && ((s >> p.page_log2) != blk || s <= before);
      const uint32_t e = __ballot_sync(0xffffffffu, ends);
      const uint32_t mine = e ? v & ((1u << (__ffs(e) - 1)) - 1u) : v;
      if (mine) {
        const int at = 31 - __clz(mine);
        last = __shfl_sync(0xffffffffu, s, at);
        len += at + 1;
        count += __popc(mine);
      }
      if (e) break;
    }
    // no token and no slot skipped: token i goes to off + i, and len <= P
    const bool dense = count == len && last - slot == len - 1;
    const int sub = lane / LPT, d0 = (lane % LPT) * 8;
    const uint8_t* x = p.x[which] + 2 * (static_cast<int64_t>(ts) * p.sx_s[which] + h * p.sx_h[which] + d0);
    const int64_t xs = 2 * p.sx_s[which];
    float amax = 0.f;
    auto largest = [&](const uint4& w) {
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack2<BF16>(ws[e]);
        const float a = fabsf(f.x), b = fabsf(f.y);
        if (a < INFINITY) amax = fmaxf(amax, a);  // NaN compares false
        if (b < INFINITY) amax = fmaxf(amax, b);
      }
    };
    uint4 held[LOADS];
    if (dense) {
#pragma unroll
      for (int k = 0; k < LOADS; ++k) {
        const int i = tw * 16 + k * TPW + sub;
        held[k] = make_uint4(0u, 0u, 0u, 0u);
        if (i < len) held[k] = *reinterpret_cast<const uint4*>(x + i * xs);
      }
#pragma unroll
      for (int k = 0; k < LOADS; ++k) largest(held[k]);
    } else {
#pragma unroll 1
      for (int i = tw * TPW + sub; i < len; i += W * TPW)
        if (valid(p.slot_map[ts + i])) largest(*reinterpret_cast<const uint4*>(x + i * xs));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float* const sp = p.scale[which] + static_cast<int64_t>(blk) * p.HKV + h;
    const float old = off > 0 ? *sp : 0.f;
    if constexpr (W > 1) {
      if (lane == 0) s_max[buf][warp] = amax;
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(W * 32) : "memory");
#pragma unroll
      for (int i = 0; i < W; ++i) amax = fmaxf(amax, s_max[buf][team * W + i]);
    } else {
      __syncwarp();  // every lane has read the old scale
    }
    float now = scale_for(amax);
    uint8_t* const y = p.cache[which] + static_cast<int64_t>(blk) * p.sc_b[which] + h * p.sc_h[which] + d0;
    const int64_t ys = p.sc_s[which];
    if (off > 0) {
      if (now > old) {  // the page's older values at the larger scale
        const float f = old / now;
#pragma unroll 2
        for (int i = tw * TPW + sub; i < off; i += W * TPW) {
          uint2* at = reinterpret_cast<uint2*>(y + i * ys);
          const uint2 w = *at;
          const uint32_t ws[2] = {w.x, w.y};
          uint32_t r[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 a = from_e4m3x2(ws[e] & 0xffffu), b = from_e4m3x2(ws[e] >> 16);
            r[e] = to_e4m3x2(a.x * f, a.y * f) | (to_e4m3x2(b.x * f, b.y * f) << 16);
          }
          *at = make_uint2(r[0], r[1]);
        }
      } else if (old >= now) {
        now = old;
      }
    }
    if (tw == 0 && lane == 0) *sp = now;
    const float inv = 1.f / now;
    const bool pow2 = (__float_as_uint(now) & 0x7fffffu) == 0;  // x * inv is then exact
    auto store = [&](int s, const uint4& w, bool exact) {
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
      uint32_t r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack2<BF16>(ws[e]);
        r[e] = exact ? to_e4m3x2(f.x * inv, f.y * inv) : to_e4m3x2(f.x / now, f.y / now);
      }
      *reinterpret_cast<uint2*>(y + s * ys) = make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
    };
    if (dense && pow2) {
#pragma unroll
      for (int k = 0; k < LOADS; ++k) {
        const int i = tw * 16 + k * TPW + sub;
        if (i < len) store(off + i, held[k], true);
      }
    } else {
#pragma unroll 1
      for (int i = tw * TPW + sub; i < len; i += W * TPW) {
        const int s = p.slot_map[ts + i];
        if (valid(s)) store(s & (P - 1), *reinterpret_cast<const uint4*>(x + i * xs), false);
      }
    }
  }
}

template <int D, bool BF16, int W>
cudaError_t launch_write_w(const KvWriteParams& p, cudaStream_t st) {
  constexpr int TEAMS = kWrThreads / 32 / W;
  const int TW = imax(1, imin(32, p.T / 512));
  const dim3 grid((p.T + TW - 1) / TW, (2 * p.HKV + TEAMS - 1) / TEAMS);
  return launch_chained(kv_write_kernel<D, BF16, W>, grid, kWrThreads, 0, st, p, TW);
}

template <int D, bool BF16>
cudaError_t launch_write_t(const KvWriteParams& p, cudaStream_t st) {
  switch (p.page_log2) {
    case 4: return launch_write_w<D, BF16, 1>(p, st);
    case 5: return launch_write_w<D, BF16, 2>(p, st);
    case 6: return launch_write_w<D, BF16, 4>(p, st);
    default: return launch_write_w<D, BF16, 8>(p, st);
  }
}

}  // namespace

cudaError_t launch_kv_tables(const KvTablesParams& p, int grid, cudaStream_t st) {
  return launch_chained(kv_tables_kernel, grid, kTabThreads, 0, st, p);
}

cudaError_t launch_kv_write(const KvWriteParams& p, bool bf16, cudaStream_t st) {
  if (p.D == 64) return bf16 ? launch_write_t<64, true>(p, st) : launch_write_t<64, false>(p, st);
  return bf16 ? launch_write_t<128, true>(p, st) : launch_write_t<128, false>(p, st);
}

}  // namespace ab
