// Attention over the paged 8-bit cache for few rows (query, head of the group)
// per KV head: single tokens, drafted tokens.
//
//   x_ij = sm_scale log2(e) ks[page j] (q_i . k_j),  p_ij = 2^(x_ij - m_i)
//   O_i  = sum_j p_ij vs[page j] v_j / l_i,  l_i = sum_j p_ij,
//   LSE_i = (m_i + log2 l_i) ln 2
//
// with k_j, v_j the stored e4m3 values, in one pass with a running m (rescaled
// only when it grows by more than 2^8).  Bound by the bytes of K and V: 2 D
// bytes and 4 D G flops a key.
//
// Split: the line of kv_sched.cuh, units of 16 rows and tiles of 64 keys, over
// persistent CTAs of 4 warps.  A warp takes 16 keys of every tile and keeps
// its own m, l and O; the four are joined in shared memory when the unit (or
// the CTA's part of it) ends.  A unit that one CTA holds whole is written at
// once; parts go to the workspace, at most two a CTA, and kv_join_kernel adds
// them in CTA order (the same result from run to run).
//
// Products: mma.m16n8k16 on fp16.  tcgen05 needs 64 or 128 rows, and here the
// group's 1 to 16 rows ride on 16, so the tensor work stays far under the time
// of the loads.  e4m3 is exact in fp16; a row of Q is brought to fp16's upper
// range by a power of two (bf16 rows keep every bit of their leading values,
// what falls under 2^-24 of fp16 is 2^-38 of the row's largest value); the
// K scale and the row's power go to the f32 score, the V scale to p before it
// is rounded to fp16, relative to the largest V scale met so far, so that
// neither scale can overflow.
//
// Layout: no operand needs a transpose through shared memory.  The sum over d
// may run in any order, so the thread that holds K column pairs c of key n in
// an mma takes 16 consecutive bytes of the key (its own cp.async of 16 bytes
// and one 16-byte read back); Q is permuted to match.  Likewise the O columns:
// the thread of column n takes bytes [n D/8, (n + 1) D/8) of its four keys, and
// two keys' bytes are paired by one byte permute before the conversion.  Each
// thread reads back only what it copied itself, so the ring needs no barrier.
#include <cuda_fp16.h>

#include "cvt.cuh"
#include "kernels.h"
#include "kv_cache.h"
#include "kv_sched.cuh"
#include "sm103.cuh"

namespace ab {

namespace {

constexpr int RT = kKvDecRows, KT = kKvDecKeys;
constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kStages = 4;       // ring of 16-key steps per warp
constexpr int kCtasPerSm = 3;
constexpr float kRescale = 8.f;  // log2 growth of a row max that triggers a rescale

template <int D>
struct DecCfg {
  static constexpr int STEP = 16 * D * 2;                       // bytes of K and V of 16 keys
  static constexpr int WARP = kStages * STEP;                   // a warp's ring
  static constexpr int JOIN = 16 * (D + 4) * 4;                 // a warp's O rows when the warps are joined
  static constexpr int REGION = WARP > JOIN ? WARP : JOIN;
  static constexpr int SMEM = kWarps * REGION + kWarps * 16 * 8;  // and its (m, l) pairs
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(in ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four e4m3 bytes -> two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t* lo, uint32_t* hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(*lo), "=r"(*hi)
      : "r"(w));
}

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Power of two that brings a largest absolute value into [2^14, 2^15), and its
// inverse; 1 for 0, infinities and NaN.
__device__ __forceinline__ float to_top(float amax, float* back) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23);  // biased
  if (!(amax > 0.f) || e == 255) {
    *back = 1.f;
    return 1.f;
  }
  int up = 14 - (e - 127);
  up = up > 126 ? 126 : up;  // subnormal rows
  *back = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
}

// Where the tile at line position ``x`` lies.
struct Cursor {
  int n, rt, h, t;
};

// Every thread of the CTA: the launch's tiles in all, and the cursor of the
// CTA's first one.  A thread sums ceil(N / 128) consecutive requests; the one
// whose requests hold the position walks them.
__device__ __forceinline__ void locate(const KvAttnParams& p, int64_t* total, int* ctas, int64_t* begin,
                                       int64_t* end, Cursor* cur) {
  __shared__ int64_t s_warp[kWarps];
  __shared__ Cursor s_cur;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = (p.N + kThreads - 1) / kThreads;
  int64_t w = 0;
  for (int i = 0; i < K; ++i) {
    const int64_t n = static_cast<int64_t>(tid) * K + i;
    if (n >= p.N) break;
    w += kv_request_tiles<RT, KT>(kv_request(static_cast<int>(n), p), p);
  }
  w *= p.HKV;
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
  *total = all;
  // no more CTAs than tiles: every CTA of a split unit then holds some of it
  const int C = all < static_cast<int64_t>(gridDim.x) ? static_cast<int>(all) : static_cast<int>(gridDim.x);
  *ctas = C;
  *begin = *end = 0;
  if (static_cast<int>(blockIdx.x) < C) {
    *begin = kv_cta_begin(all, blockIdx.x, C);
    *end = kv_cta_begin(all, blockIdx.x + 1, C);
  }
  int64_t x = *begin - (base + inc - w);  // relative to my requests
  if (*begin < *end && x >= 0 && x < w) {
    for (int n = tid * K;; ++n) {
      const KvReq r = kv_request(n, p);
      const int64_t wn = kv_request_tiles<RT, KT>(r, p) * p.HKV;
      if (x >= wn) {
        x -= wn;
        continue;
      }
      for (int rt = 0;; ++rt) {
        const KvTiles k = kv_row_tile<RT, KT>(r, rt, p);
        const int64_t wr = static_cast<int64_t>(k.n) * p.HKV;
        if (x >= wr) {
          x -= wr;
          continue;
        }
        s_cur = Cursor{n, rt, static_cast<int>(x / k.n), static_cast<int>(x % k.n)};
        break;
      }
      break;
    }
  }
  __syncthreads();
  *cur = s_cur;
}

// Writes of one row's final O (16-bit, ND values from column d0) and LSE.
template <bool BF16, int ND>
__device__ __forceinline__ void store_o(const KvAttnParams& p, int64_t t, int hq, int d0, const float* o) {
  uint8_t* out = p.o + 2 * (t * p.so_s + static_cast<int64_t>(hq) * p.so_h + d0);
  if constexpr (ND >= 8) {
#pragma unroll
    for (int i = 0; i < ND; i += 8) {
      uint4 w;
      w.x = pack2<BF16>(o[i], o[i + 1]), w.y = pack2<BF16>(o[i + 2], o[i + 3]);
      w.z = pack2<BF16>(o[i + 4], o[i + 5]), w.w = pack2<BF16>(o[i + 6], o[i + 7]);
      *reinterpret_cast<uint4*>(out + 2 * i) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < ND; i += 2) *reinterpret_cast<uint32_t*>(out + 2 * i) = pack2<BF16>(o[i], o[i + 1]);
  }
}

// m in log2 units; a row that saw no key has l = 0.
__device__ __forceinline__ void store_lse(const KvAttnParams& p, int64_t t, int hq, float m, float l) {
  p.lse[hq * p.sl_h + t * p.sl_s] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv_decode_kernel(const KvAttnParams p) {
  using C = DecCfg<D>;
  constexpr int KC = D / 64;   // 16-byte chunks of a key's row per thread
  constexpr int VB = D / 8;    // bytes of a value row per thread
  constexpr int NT = D / 8;    // column tiles of O
  extern __shared__ __align__(16) uint8_t sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r8 = lane >> 2, c4 = lane & 3;
  uint8_t* const ring = sm + warp * C::REGION;
  const uint32_t ring_s = smem_u32(ring);
  float2* const ml = reinterpret_cast<float2*>(sm + kWarps * C::REGION);  // [warp][16]

  grid_dependency_wait();
  if (blockIdx.x == 0 && tid == 0) *p.err = 0;
  int64_t total, begin, end;
  int ctas;
  Cursor cur;
  locate(p, &total, &ctas, &begin, &end, &cur);
  if (tid == 0) p.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (begin >= end) return;

  KvReq rq = kv_request(cur.n, p);
  for (int64_t x = begin; x < end;) {
    // ---------------------------------------------------------- the unit and the CTA's part of it
    const KvTiles kt = kv_row_tile<RT, KT>(rq, cur.rt, p);
    const int part0 = cur.t;
    const int64_t left = end - x;
    const int part1 = kt.n - part0 <= left ? kt.n : part0 + static_cast<int>(left);
    const int row0 = cur.rt * RT;
    const int rows = imin(RT, rq.R - row0);
    // my two rows: their queries and key ranges, and Q in fp16
    int lo[2], hi[2];
    float rs[2];
    uint32_t qa[KC * 4][4];  // [k step][a0..a3]
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = r8 + 8 * e;
      const bool live = r < rows;
      const int i = (row0 + r) / p.G, g = (row0 + r) % p.G;
      lo[e] = hi[e] = 0;
      if (live) kv_row_keys(rq, i, p.causal, p.window, &lo[e], &hi[e]);
      const uint8_t* src = p.q + 2 * ((static_cast<int64_t>(rq.a) + i) * p.sq_s +
                                      static_cast<int64_t>(cur.h * p.G + g) * p.sq_h);
      uint32_t w[KC][8];
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint4 x4 = make_uint4(0u, 0u, 0u, 0u);
          if (live) x4 = *reinterpret_cast<const uint4*>(src + 2 * (c * 64 + c4 * 16 + u * 8));
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
      rs[e] = back * p.scale_log2;
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float2 f = unpack2<BF16>(w[c][u]);
          // bytes 4j .. 4j + 3 of the chunk are k step 4c + j: pairs (0,1) and (2,3)
          qa[c * 4 + u / 2][e + 2 * (u & 1)] = pack2<false>(f.x * up, f.y * up);
        }
    }
    // keys that every live row sees lie in [lo_all, hi_all)
    int lo_all, hi_all, xx;
    kv_row_keys(rq, (row0 + rows - 1) / p.G, p.causal, p.window, &lo_all, &xx);
    kv_row_keys(rq, row0 / p.G, p.causal, p.window, &xx, &hi_all);

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, vref = 0.f, vinv = 0.f;
    float o[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

    // Page ids of my steps, 32 tiles at a time: lane i holds those of tile
    // ``batch + i``; scales likewise.
    const uint8_t* const kh = p.k + static_cast<int64_t>(cur.h) * p.sk_h;
    const uint8_t* const vh = p.v + static_cast<int64_t>(cur.h) * p.sv_h;
    int ld_batch = part0, blk_l = -1;
    auto key0_of = [&](int t) { return (kt.t0 + t) * KT + warp * 16; };
    auto load_ids = [&](int batch) {
      const int t = batch + lane;
      int b = -1;
      if (t < part1) {
        const int k0 = key0_of(t);
        if (k0 < kt.hi && k0 + 16 > kt.lo) {
          b = p.table[cur.n * p.table_stride + (k0 >> p.page_log2)];
          if (b < 0 || b >= p.num_blocks) b = -1;
        }
      }
      blk_l = b;
    };
    load_ids(part0);
    float ks_l = 0.f, vs_l = 0.f;  // scales of the batch being computed
    int cp_blk = -1;               // its ids (the load side may be a batch ahead)
    auto issue = [&](int t) {  // copies of tile t's 16 keys into stage t % kStages
      if (t - ld_batch == 32) {
        ld_batch += 32;
        load_ids(ld_batch);
      }
      if (t < part1) {
        const int b = __shfl_sync(0xffffffffu, blk_l, t - ld_batch);
        const uint32_t dst = ring_s + ((t - part0) % kStages) * C::STEP;
        const bool in = b >= 0;
        const int s0 = key0_of(t) & ((1 << p.page_log2) - 1);
        const int64_t bb = in ? b : 0;
        const uint8_t* ks = kh + bb * p.sk_b + (in ? s0 : 0) * p.sk_s;
        const uint8_t* vs = vh + bb * p.sv_b + (in ? s0 : 0) * p.sv_s;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < KC; ++c)
            cp16(dst + ((j * KC + c) * 32 + lane) * 16, ks + (j * 8 + r8) * p.sk_s + c * 64 + c4 * 16, in);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = 2 * c4 + (e & 1) + 8 * (e >> 1);
          const uint32_t d = dst + 16 * D + (e * 32 + lane) * VB;
          if constexpr (VB == 16)
            cp16(d, vs + key * p.sv_s + r8 * VB, in);
          else
            cp8(d, vs + key * p.sv_s + r8 * VB, in);
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(part0 + i);

    int cp_batch = part0 - 32;
    for (int t = part0; t < part1; ++t) {
      if (t - cp_batch == 32) {
        // scales of the next 32 tiles (their ids once more: the load side may
        // have moved on)
        cp_batch = t;
        const int u = t + lane;
        cp_blk = -1, ks_l = vs_l = 0.f;
        if (u < part1) {
          const int k0 = key0_of(u);
          if (k0 < kt.hi && k0 + 16 > kt.lo) {
            const int b = p.table[cur.n * p.table_stride + (k0 >> p.page_log2)];
            if (b >= 0 && b < p.num_blocks) {
              cp_blk = b;
              const int64_t at = static_cast<int64_t>(b) * p.HKV + cur.h;
              ks_l = p.k_scale[at];
              vs_l = p.v_scale[at] < 0x1p-126f ? 0.f : p.v_scale[at];  // (its inverse is taken)
            }
          }
        }
      }
      cp_wait<kStages - 2>();
      issue(t + kStages - 1);
      const int bi = t - cp_batch;
      const float ks = __shfl_sync(0xffffffffu, ks_l, bi), vs = __shfl_sync(0xffffffffu, vs_l, bi);
      if (__shfl_sync(0xffffffffu, cp_blk, bi) < 0) continue;
      const uint8_t* const st = ring + ((t - part0) % kStages) * C::STEP;
      const int k0 = key0_of(t);

      // ---- scores of 16 keys
      float s[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const uint4 w = *reinterpret_cast<const uint4*>(st + ((j * KC + c) * 32 + lane) * 16);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t b0, b1;
            e4m3x4_to_f16(ww[u], &b0, &b1);
            mma16816(s[j], qa[c * 4 + u], b0, b1);
          }
        }
      }
      const bool edge = k0 < lo_all || k0 + 16 > hi_all;
      const float f0 = ks * rs[0], f1 = ks * rs[1];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        s[j][0] *= f0, s[j][1] *= f0, s[j][2] *= f1, s[j][3] *= f1;
        if (edge) {
          const int k = k0 + j * 8 + 2 * c4;
          if (k < lo[0] || k >= hi[0]) s[j][0] = -INFINITY;
          if (k + 1 < lo[0] || k + 1 >= hi[0]) s[j][1] = -INFINITY;
          if (k < lo[1] || k >= hi[1]) s[j][2] = -INFINITY;
          if (k + 1 < lo[1] || k + 1 >= hi[1]) s[j][3] = -INFINITY;
        }
      }
      // ---- running max, lazily adopted; the V scale's reference likewise
      float mx0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float mx1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
      // (a row without a key yet has m = -inf and adopts any finite max)
      const bool up0 = mx0 > m[0] + kRescale, up1 = mx1 > m[1] + kRescale;
      if (__any_sync(0xffffffffu, up0 || up1 || vs > vref)) {
        const float a0 = up0 ? ex2(m[0] - mx0) : 1.f, a1 = up1 ? ex2(m[1] - mx1) : 1.f;  // ex2(-inf) = 0
        if (up0) m[0] = mx0;
        if (up1) m[1] = mx1;
        float g = 1.f;
        if (vs > vref) {
          g = vref / vs;
          vref = vs;
          vinv = 1.f / vs;
        }
        l[0] *= a0, l[1] *= a1;
        const float g0 = a0 * g, g1 = a1 * g;
#pragma unroll
        for (int u = 0; u < NT; ++u) o[u][0] *= g0, o[u][1] *= g0, o[u][2] *= g1, o[u][3] *= g1;
      }
      const float ratio = vs * vinv;  // at most 1
      const float n0 = m[0] == -INFINITY ? 0.f : m[0], n1 = m[1] == -INFINITY ? 0.f : m[1];
      uint32_t pa[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float p0 = ex2(s[j][0] - n0), p1 = ex2(s[j][1] - n0), p2 = ex2(s[j][2] - n1), p3 = ex2(s[j][3] - n1);
        l[0] += p0 + p1;
        l[1] += p2 + p3;
        pa[2 * j] = pack2<false>(p0 * ratio, p1 * ratio);
        pa[2 * j + 1] = pack2<false>(p2 * ratio, p3 * ratio);
      }
      // ---- O += P V
      constexpr int VW = VB / 4;
      uint32_t vw[4][VW];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint8_t* at = st + 16 * D + (e * 32 + lane) * VB;
        if constexpr (VB == 16) {
          const uint4 w = *reinterpret_cast<const uint4*>(at);
          vw[e][0] = w.x, vw[e][1] = w.y, vw[e][2] = w.z, vw[e][3] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(at);
          vw[e][0] = w.x, vw[e][1] = w.y;
        }
        if (edge) {  // a zero P times a NaN byte would be NaN: keys that no row sees are zeroed
          const int k = k0 + 2 * c4 + (e & 1) + 8 * (e >> 1);
          if (k < kt.lo || k >= kt.hi) {
#pragma unroll
            for (int u = 0; u < VW; ++u) vw[e][u] = 0u;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < VW; ++u) {
        // bytes 4u .. 4u + 3 of keys (0, 1) and (2, 3) paired: columns 4u .. 4u + 3
        uint32_t b[4][2];
        e4m3x4_to_f16(__byte_perm(vw[0][u], vw[1][u], 0x5140), &b[0][0], &b[1][0]);
        e4m3x4_to_f16(__byte_perm(vw[0][u], vw[1][u], 0x7362), &b[2][0], &b[3][0]);
        e4m3x4_to_f16(__byte_perm(vw[2][u], vw[3][u], 0x5140), &b[0][1], &b[1][1]);
        e4m3x4_to_f16(__byte_perm(vw[2][u], vw[3][u], 0x7362), &b[2][1], &b[3][1]);
#pragma unroll
        for (int y = 0; y < 4; ++y) mma16816(o[u * 4 + y], pa, b[y][0], b[y][1]);
      }
    }
    cp_wait<0>();  // (the last groups are empty) the ring is free

    // ---------------------------------------------------------- the warps joined
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    // every lane has read its last stage before the warp's region is reused
    __syncwarp();
    float* const jo = reinterpret_cast<float*>(ring);
    // O rows of D + 4 floats; column 2 c4 e' of tile u is d = (2 c4 + e') D/8 + u
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int u = 0; u < NT; u += 4) {
          float4 w = make_float4(o[u][2 * e + y], o[u + 1][2 * e + y], o[u + 2][2 * e + y], o[u + 3][2 * e + y]);
          w.x *= vref, w.y *= vref, w.z *= vref, w.w *= vref;
          *reinterpret_cast<float4*>(jo + (r8 + 8 * e) * (D + 4) + (2 * c4 + y) * NT + u) = w;
        }
    if (c4 == 0) {
      ml[warp * 16 + r8] = make_float2(m[0], l[0]);
      ml[warp * 16 + r8 + 8] = make_float2(m[1], l[1]);
    }
    __syncthreads();
    const bool whole = part0 == 0 && part1 == kt.n;
    const int slot = 2 * blockIdx.x + (part0 > 0 ? 0 : 1);
    constexpr int ND = D / 8;  // columns a thread joins: 8 threads a row
    const int row = tid >> 3, d0 = (tid & 7) * ND;
    if (row < rows) {
      float mm = -INFINITY, w[kWarps], ll = 0.f, acc[ND];
#pragma unroll
      for (int i = 0; i < kWarps; ++i) mm = fmaxf(mm, ml[i * 16 + row].x);
#pragma unroll
      for (int u = 0; u < ND; ++u) acc[u] = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float2 v = ml[i * 16 + row];
        w[i] = v.y == 0.f ? 0.f : ex2(v.x - mm);
        ll += w[i] * v.y;
        const float* from = reinterpret_cast<const float*>(sm + i * C::REGION) + row * (D + 4) + d0;
        if (v.y != 0.f) {
#pragma unroll
          for (int u = 0; u < ND; u += 4) {
            const float4 f = *reinterpret_cast<const float4*>(from + u);
            acc[u] += w[i] * f.x, acc[u + 1] += w[i] * f.y, acc[u + 2] += w[i] * f.z, acc[u + 3] += w[i] * f.w;
          }
        }
      }
      if (whole) {
        const int i = (row0 + row) / p.G, hq = cur.h * p.G + (row0 + row) % p.G;
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
        for (int u = 0; u < ND; ++u) acc[u] *= inv;
        store_o<BF16, ND>(p, static_cast<int64_t>(rq.a) + i, hq, d0, acc);
        if (d0 == 0) store_lse(p, static_cast<int64_t>(rq.a) + i, hq, mm, ll);
      } else {
        float* to = p.part_o + (static_cast<int64_t>(slot) * RT + row) * D + d0;
#pragma unroll
        for (int u = 0; u < ND; u += 4)
          *reinterpret_cast<float4*>(to + u) = make_float4(acc[u], acc[u + 1], acc[u + 2], acc[u + 3]);
        if (d0 == 0) p.part_ml[slot * RT + row] = make_float2(mm, ll);
      }
    }
    if (tid == 0 && part0 > 0 && part1 == kt.n) {
      // this part ends a unit that CTA c0 began
      const int c0 = kv_cta_of(total, begin - part0, ctas);
      p.desc[blockIdx.x] = make_int4(cur.n, cur.rt, cur.h, c0);
    }
    __syncthreads();  // the joined rows are read before the ring fills again

    // ---------------------------------------------------------- next unit
    x += part1 - part0;
    cur.t = 0;
    if (x < end && ++cur.h == p.HKV) {
      cur.h = 0;
      if (++cur.rt == kv_row_tiles<RT>(rq)) {
        cur.rt = 0;
        do {
          rq = kv_request(++cur.n, p);
        } while (rq.R == 0);
      }
    }
  }
}

// Joins the parts of each unit that was split over CTAs: block c the unit that
// CTA c finished (a CTA finishes at most one that it did not begin), its parts
// from c0 (which began it) to c in order.  A warp a row: lanes first take the
// parts' (m, l) together, then D/32 columns each.
template <int D, bool BF16>
__global__ void __launch_bounds__(RT * 32) kv_join_kernel(const KvAttnParams p) {
  grid_dependency_wait();
  const int c = blockIdx.x, row = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 d = p.desc[c];
  if (d.x < 0) return;
  const KvReq rq = kv_request(d.x, p);
  const int row0 = d.y * RT;
  if (row0 + row >= rq.R) return;
  const int c0 = d.w, parts = c - c0 + 1;
  auto slot_of = [&](int i) { return 2 * (c0 + i) + (i == 0 ? 1 : 0); };
  float m = -INFINITY;
  for (int i = lane; i < parts; i += 32) m = fmaxf(m, p.part_ml[slot_of(i) * RT + row].x);
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  constexpr int ND = D / 32;
  float acc[ND], l = 0.f;
#pragma unroll
  for (int u = 0; u < ND; ++u) acc[u] = 0.f;
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float w = 0.f;
    if (i0 + lane < parts) {
      const float2 v = p.part_ml[slot_of(i0 + lane) * RT + row];
      w = v.y == 0.f ? 0.f : ex2(v.x - m);
      l += w * v.y;
    }
    const int n = imin(32, parts - i0);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float f = __shfl_sync(0xffffffffu, w, i);
      const float* from = p.part_o + (static_cast<int64_t>(slot_of(i0 + i)) * RT + row) * D + lane * ND;
      float v[ND];
      if constexpr (ND == 4) {
        const float4 x = *reinterpret_cast<const float4*>(from);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(from);
        v[0] = x.x, v[1] = x.y;
      }
#pragma unroll
      for (int u = 0; u < ND; ++u) acc[u] += f != 0.f ? f * v[u] : 0.f;
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
  const int i = (row0 + row) / p.G, hq = d.z * p.G + (row0 + row) % p.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int u = 0; u < ND; ++u) acc[u] *= inv;
  store_o<BF16, ND>(p, static_cast<int64_t>(rq.a) + i, hq, lane * ND, acc);
  if (lane == 0) store_lse(p, static_cast<int64_t>(rq.a) + i, hq, m, l);
}

template <int D, bool BF16>
cudaError_t launch_t(const KvAttnParams& p, int sms, cudaStream_t st) {
  auto kern = kv_decode_kernel<D, BF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, DecCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = imin(sms * kCtasPerSm, kKvDecMaxCtas);
  e = launch_after_previous(kern, grid, kThreads, DecCfg<D>::SMEM, st, p);
  if (e != cudaSuccess) return e;
  return launch_after_previous(kv_join_kernel<D, BF16>, grid, RT * 32, 0, st, p);
}

}  // namespace

cudaError_t launch_kv_decode(const KvAttnParams& p, bool bf16, int sms, cudaStream_t st) {
  if (p.D == 64) return bf16 ? launch_t<64, true>(p, sms, st) : launch_t<64, false>(p, sms, st);
  return bf16 ? launch_t<128, true>(p, sms, st) : launch_t<128, false>(p, sms, st);
}

}  // namespace ab
