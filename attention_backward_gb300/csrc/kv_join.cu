// The second launch of attention over the cache: rows whose keys were split
// over workers are joined from their f32 partials in the workspace.
#include "cvt.cuh"
#include "kv_cache.h"
#include "kv_common.cuh"
#include "kv_launch.h"
#include "sm103.cuh"

namespace ab {

namespace {

// Joins the parts of each unit that was split over workers: entry w of ``desc``
// (first row of q of the request, first row of the unit in the request, head and
// rows, first part) names the unit that worker w finished (a worker finishes at most one that it
// did not begin), its parts d.w to w / stride in order; d.w is -1 where there is
// none.  stride: workers per part (one a head in kv_decode.cu, 1
// in kv_prompt.cu).  Every block lists the finished units (a scan of all
// entries); their rows are then spread over all warps of the launch,
// with as many warps a row as there are to spare.  These add fixed shares of
// the parts in order: lanes first take the parts' (m, l) together, then D/32
// columns each.  Latency-bound: a few parts a unit as a rule, hundreds where few
// requests have all the workers: 5 to 8 us for units of few rows, 15 us for 151
// units of 256 rows of 128.
constexpr int kJoinWarps = 16;

template <int D, int RT, bool BF16>
__device__ __forceinline__ void join_units(const KvAttnParams& p, const KvJoinPart& from, int block, int blocks,
                                           int4* list, float (*s_o)[D], float2* s_ml, int* s_cnt) {
  constexpr int ND = D / 32, PER = kKvDecMaxWorkers / (kJoinWarps * 32);
  // Rows of a warp at once, and parts in flight: parts may be many where units are
  // of few rows, and are two or three as a rule where they are of 256 (two or four
  // rows at once take 15 us on 3761 prompt tokens, eight 18; eight parts in flight
  // instead of four take 1 us more on 32 requests of drafted tokens).
  constexpr int NR = RT > 16 ? 4 : 1, PF = RT > 16 ? 1 : 4;
  const int workers = from.workers, stride = from.stride;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int4 d[PER];  // of workers tid * PER + i
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    d[i] = make_int4(0, 0, 0, -1);
    if (tid * PER + i < workers) d[i] = from.desc[tid * PER + i];
  }
  int mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) mine += d[i].w >= 0 ? 1 : 0;
  int at0 = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, at0, s);
    if (lane >= s) at0 += v;
  }
  if (lane == 31) s_cnt[warp] = at0;
  __syncthreads();
  at0 -= mine;
  int units = 0;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) {
    if (i < warp) at0 += s_cnt[i];
    units += s_cnt[i];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (d[i].w >= 0) list[at0++] = make_int4(d[i].x, d[i].y, d[i].z, d[i].w << 16 | ((tid * PER + i) / stride - d[i].w + 1));
  __syncthreads();
  const int items = units * (RT / NR);  // those past a unit's last row are skipped
  int ls = 0;                           // log2 of the warps an item
  if (NR == 1)
    while ((1 << ls) < kJoinWarps && items << (ls + 1) <= blocks * kJoinWarps) ++ls;
  const int shares = NR == 1 ? 1 << ls : 1;
  const int group = warp >> ls, share = warp & (shares - 1), groups = kJoinWarps >> ls;
  for (int t0 = block * groups; t0 < items; t0 += blocks * groups) {
    const int item = t0 + group;
    int4 u = make_int4(0, 0, 0, 0);
    int head = 0, live = 0, i0 = 0, i1 = 0;
    const int row = item % (RT / NR) * NR;  // my first row of the unit
    if (item < items) {
      u = list[item / (RT / NR)];
      head = u.z >> 16, live = u.z & 0xffff;
      const int parts = u.w & 0xffff;
      i0 = parts * share >> ls, i1 = parts * (share + 1) >> ls;
    }
    const int g0 = u.w >> 16;  // its first part
    auto slot_of = [&](int i) { return 2 * ((g0 + i) * stride + (stride > 1 ? head : 0)) + (i == 0 ? 1 : 0); };
    float m[NR], acc[NR][ND], l = 0.f;  // l: my lane's share of row lane % NR's
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      m[r] = -INFINITY;
#pragma unroll
      for (int u = 0; u < ND; ++u) acc[r][u] = 0.f;
    }
    if (row < live) {
      // PF parts of NR rows in flight; (m, l) of up to 32 / NR parts looked up together, a lane each
      constexpr int LOOK = 32 / NR;
      for (int j = i0; j < i1; j += LOOK) {
        const int n = imin(LOOK, i1 - j);
        float2 v = make_float2(0.f, 0.f);
        if (lane / NR < n && row + lane % NR < live) v = from.part_ml[static_cast<int64_t>(slot_of(j + lane / NR)) * RT + row + lane % NR];
        float x[PF][NR][ND];
        auto load = [&](int i) {  // PF parts' rows from part i on
#pragma unroll
          for (int k = 0; k < PF; ++k) {
            const int64_t at = static_cast<int64_t>(slot_of(j + imin(i + k, n - 1))) * RT + row;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const float* src = from.part_o + (at + imin(r, live - 1 - row)) * D + lane * ND;
              if constexpr (ND == 4) {
                const float4 y = *reinterpret_cast<const float4*>(src);
                x[k][r][0] = y.x, x[k][r][1] = y.y, x[k][r][2] = y.z, x[k][r][3] = y.w;
              } else {
                const float2 y = *reinterpret_cast<const float2*>(src);
                x[k][r][0] = y.x, x[k][r][1] = y.y;
              }
            }
          }
        };
        load(0);  // (in flight while the weights are made)
        // the rows' max over these parts (lanes of one row are NR apart), then their weights
        float mx = v.y == 0.f ? -INFINITY : v.x;
#pragma unroll
        for (int s = NR; s < 32; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
        float mine_m = m[0];
#pragma unroll
        for (int r = 1; r < NR; ++r) mine_m = lane % NR == r ? m[r] : mine_m;
        mx = fmaxf(mx, mine_m);  // of row lane % NR
        const float w = v.y == 0.f ? 0.f : ex2(v.x - mx);
        l = (mine_m == mx ? l : (mine_m == -INFINITY ? 0.f : l * ex2(mine_m - mx))) + w * v.y;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float mr = __shfl_sync(0xffffffffu, mx, r);
          const float g = m[r] == mr ? 1.f : (m[r] == -INFINITY ? 0.f : ex2(m[r] - mr));
          m[r] = mr;
#pragma unroll
          for (int u = 0; u < ND; ++u) acc[r][u] *= g;
        }
        for (int i = 0; i < n; i += PF) {
          if (i > 0) load(i);
#pragma unroll
          for (int k = 0; k < PF; ++k)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const float f = __shfl_sync(0xffffffffu, w, ((i + k) * NR + r) & 31);
              if (i + k < n && f != 0.f) {  // (a part that saw no key of the row says nothing)
#pragma unroll
                for (int u = 0; u < ND; ++u) acc[r][u] += f * x[k][r][u];
              }
            }
        }
      }
#pragma unroll
      for (int s = 16; s >= NR; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
      if (share > 0) {
#pragma unroll
        for (int u = 0; u < ND; ++u) s_o[NR == 1 ? warp : 0][lane * ND + u] = acc[0][u];
        if (lane == 0) s_ml[warp] = make_float2(m[0], l);
      }
    }
    if (shares > 1) __syncthreads();
    if (share == 0 && row < live) {
      int i = (u.y + row) / p.G, h = (u.y + row) % p.G;  // query and head of the group of my first row
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        if (row + r >= live) break;
        float lr = NR == 1 ? l : __shfl_sync(0xffffffffu, l, r);
        if constexpr (NR == 1) {
          for (int k = 1; k < shares; ++k) {
            const float2 v = s_ml[warp + k];
            if (v.y == 0.f) continue;
            const float mx = fmaxf(m[r], v.x), g = lr == 0.f ? 0.f : ex2(m[r] - mx), f = ex2(v.x - mx);
            lr = lr * g + v.y * f;
            m[r] = mx;
#pragma unroll
            for (int u = 0; u < ND; ++u) acc[r][u] = acc[r][u] * g + s_o[warp + k][lane * ND + u] * f;
          }
        }
        const int64_t at = static_cast<int64_t>(u.x) + i;
        const int hq = head * p.G + h;
        const float inv = lr == 0.f ? 0.f : 1.f / lr;
#pragma unroll
        for (int u = 0; u < ND; ++u) acc[r][u] *= inv;
        store_o<BF16, ND>(p, at, hq, lane * ND, acc[r]);
        if (lane == 0) store_lse(p, at, hq, m[r], lr);
        if (++h == p.G) h = 0, ++i;
      }
    }
    if (shares > 1) __syncthreads();
  }
}

// The first ``blocks_a`` blocks join the units of a, of RT rows, the others those
// of b, of kKvPrRows (a batch of few and many rows: both kernels' in one launch).
template <int D, int RT, bool BF16>
__global__ void __launch_bounds__(kJoinWarps * 32, 2)
    kv_join_kernel(const KvAttnParams p, const KvJoinPart a, const KvJoinPart b, int blocks_a) {
  __shared__ int4 list[kKvDecMaxWorkers];  // entries, their parts in place of the first part's number
  __shared__ int s_cnt[kJoinWarps];
  __shared__ float s_o[RT > 16 ? 1 : kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  grid_dependency_wait();
  const int tid = threadIdx.x, block = blockIdx.x;
  int err = kErrNone;  // (no kernel has more CTAs than a block has threads)
  if (block == 0) {
    if (tid < b.ctas) err = b.cta_err[tid];
    if (tid < a.ctas && a.cta_err[tid] != kErrNone) err = a.cta_err[tid];
  }
  if (RT > 16 || block < blocks_a)
    join_units<D, RT, BF16>(p, a, block, blocks_a, list, s_o, s_ml, s_cnt);
  else
    join_units<D, kKvPrRows, BF16>(p, b, block - blocks_a, gridDim.x - blocks_a, list, s_o, s_ml, s_cnt);
  if (block == 0) {  // the call's error word: some CTA's error, if there is any
    if (tid == 0) *p.err = kErrNone;
    if (__syncthreads_or(err != kErrNone) && err != kErrNone) *p.err = err;
  }
}

template <int D, bool BF16>
cudaError_t launch_rt(const KvAttnParams& p, int rt, const KvJoinPart& a, const KvJoinPart& b, int sms,
                      cudaStream_t st) {
  auto kern = rt == 8 ? kv_join_kernel<D, 8, BF16> : rt == 16 ? kv_join_kernel<D, 16, BF16> : kv_join_kernel<D, kKvPrRows, BF16>;
  return launch_chained(kern, 2 * sms, kJoinWarps * 32, 0, st, p, a, b, b.workers > 0 ? sms : 2 * sms);
}

}  // namespace

cudaError_t launch_kv_join(const KvAttnParams& p, bool bf16, const KvJoinPart& few, const KvJoinPart& many, int sms,
                           cudaStream_t st) {
  const bool both = few.workers > 0 && many.workers > 0;
  const KvJoinPart &a = few.workers > 0 ? few : many, b = both ? many : KvJoinPart{};
  const int rt = few.workers > 0 ? few.rows : kKvPrRows;
  if (p.D == 64)
    return bf16 ? launch_rt<64, true>(p, rt, a, b, sms, st) : launch_rt<64, false>(p, rt, a, b, sms, st);
  return bf16 ? launch_rt<128, true>(p, rt, a, b, sms, st) : launch_rt<128, false>(p, rt, a, b, sms, st);
}

}  // namespace ab
