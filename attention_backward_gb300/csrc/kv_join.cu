// The second launch of attention over the cache: rows whose keys were split
// over workers are joined from their f32 partials in the workspace.
#include "cvt.cuh"
#include "kernels.h"
#include "kv_cache.h"
#include "kv_common.cuh"
#include "kv_sched.cuh"
#include "sm103.cuh"

namespace ab {

namespace {

// Joins the parts of each unit that was split over workers: entry w of ``desc``
// names the unit that worker w finished (a worker finishes at most one that it
// did not begin), its parts d.w to w / stride in order; ``fin`` holds d.w, or -1
// where there is none.  stride: workers per part (one a head in kv_decode.cu, 1
// in kv_prompt.cu).  Every block lists the finished units (a scan of one
// flag a worker); their rows are then spread over all warps of the launch,
// with as many warps a row as there are to spare.  These add fixed shares of
// the parts in order: lanes first take the parts' (m, l) together, then D/32
// columns each.  Latency-bound: a few parts a unit as a rule, hundreds where few
// requests have all the workers.
constexpr int kJoinWarps = 16;

template <int D, int RT, bool BF16>
__global__ void __launch_bounds__(kJoinWarps * 32, 2) kv_join_kernel(const KvAttnParams p, int workers, int ctas, int stride,
                                                                  bool first) {
  constexpr int ND = D / 32, PER = kKvDecMaxWorkers / (kJoinWarps * 32);
  __shared__ uint16_t list[kKvDecMaxWorkers];
  __shared__ int s_cnt[kJoinWarps];
  __shared__ float s_o[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  grid_dependency_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x == 0 && warp == 0) {  // the launch's error word
    int e = kErrNone;
    for (int i = lane; i < ctas; i += 32) e = imax(e, p.cta_err[i]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) e = imax(e, __shfl_xor_sync(0xffffffffu, e, s));
    if (lane == 0) *p.err = first ? e : imax(e, *p.err);
  }
  uint32_t mine = 0;  // my PER workers that finished a unit
#pragma unroll
  for (int i = 0; i < PER; i += 4) {
    const int w = tid * PER + i;
    if (w < workers) {  // (the flags' space is a multiple of 16 bytes)
      const int4 f = *reinterpret_cast<const int4*>(p.fin + w);
      mine |= ((f.x >= 0 ? 1u : 0u) | (f.y >= 0 && w + 1 < workers ? 2u : 0u) | (f.z >= 0 && w + 2 < workers ? 4u : 0u) |
               (f.w >= 0 && w + 3 < workers ? 8u : 0u))
              << i;
    }
  }
  int at0 = __popc(mine);
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, at0, s);
    if (lane >= s) at0 += v;
  }
  if (lane == 31) s_cnt[warp] = at0;
  __syncthreads();
  at0 -= __popc(mine);
  int units = 0;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) {
    if (i < warp) at0 += s_cnt[i];
    units += s_cnt[i];
  }
  for (uint32_t m = mine; m != 0; m &= m - 1) list[at0++] = static_cast<uint16_t>(tid * PER + __ffs(m) - 1);
  __syncthreads();
  const int rows = units * RT;  // those past a unit's last row are skipped
  int shares = 1;               // warps a row
  while (shares < kJoinWarps && rows * shares * 2 <= static_cast<int>(gridDim.x) * kJoinWarps) shares *= 2;
  const int group = warp / shares, share = warp % shares, groups = kJoinWarps / shares;
  for (int r0 = blockIdx.x * groups; r0 < rows; r0 += static_cast<int>(gridDim.x) * groups) {
    const int item = r0 + group;
    KvReq rq{};
    int4 d = make_int4(-1, 0, 0, 0);
    int row0 = 0, live = 0, i0 = 0, i1 = 0;
    const int row = item % RT;
    if (item < rows) {
      const int w = list[item / RT];
      d = p.desc[w];
      rq = kv_request(d.x, p);
      row0 = d.y * RT, live = imin(RT, rq.R - row0);
      const int parts = w / stride - d.w + 1;
      i0 = parts * share / shares, i1 = parts * (share + 1) / shares;
    }
    auto slot_of = [&](int i) { return 2 * ((d.w + i) * stride + (stride > 1 ? d.z : 0)) + (i == 0 ? 1 : 0); };
    float m = -INFINITY, l = 0.f, acc[ND];
#pragma unroll
    for (int u = 0; u < ND; ++u) acc[u] = 0.f;
    if (row < live) {
      for (int j = i0; j < i1; j += 32) {
        // (m, l) of up to 32 parts, then their rows, rescaled where m grows
        const float2 v = j + lane < i1 ? p.part_ml[slot_of(j + lane) * RT + row] : make_float2(0.f, 0.f);
        float mx = v.y == 0.f ? -INFINITY : v.x;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
        mx = fmaxf(mx, m);
        if (mx > m) {
          const float g = m == -INFINITY ? 0.f : ex2(m - mx);
          l *= g;
#pragma unroll
          for (int u = 0; u < ND; ++u) acc[u] *= g;
          m = mx;
        }
        const float f = v.y == 0.f ? 0.f : ex2(v.x - m);
        l += f * v.y;
        const int n = imin(32, i1 - j);
        for (int i = 0; i < n; i += 8) {  // eight rows in flight
          float x[8][ND];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int at = slot_of(j + imin(i + k, n - 1));
            const float* from = p.part_o + (static_cast<int64_t>(at) * RT + row) * D + lane * ND;
            if constexpr (ND == 4) {
              const float4 y = *reinterpret_cast<const float4*>(from);
              x[k][0] = y.x, x[k][1] = y.y, x[k][2] = y.z, x[k][3] = y.w;
            } else {
              const float2 y = *reinterpret_cast<const float2*>(from);
              x[k][0] = y.x, x[k][1] = y.y;
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, (i + k) & 31);
            if (i + k < n && fk != 0.f) {  // (a part that saw no key of the row says nothing)
#pragma unroll
              for (int u = 0; u < ND; ++u) acc[u] += fk * x[k][u];
            }
          }
        }
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
      if (share > 0) {
#pragma unroll
        for (int u = 0; u < ND; ++u) s_o[warp][lane * ND + u] = acc[u];
        if (lane == 0) s_ml[warp] = make_float2(m, l);
      }
    }
    if (shares > 1) __syncthreads();
    if (share == 0 && row < live) {
      for (int k = 1; k < shares; ++k) {
        const float2 v = s_ml[warp + k];
        if (v.y == 0.f) continue;
        const float mx = fmaxf(m, v.x), g = l == 0.f ? 0.f : ex2(m - mx), f = ex2(v.x - mx);
        l = l * g + v.y * f;
        m = mx;
#pragma unroll
        for (int u = 0; u < ND; ++u) acc[u] = acc[u] * g + s_o[warp + k][lane * ND + u] * f;
      }
      const int64_t at = static_cast<int64_t>(rq.a) + (row0 + row) / p.G;
      const int hq = d.z * p.G + (row0 + row) % p.G;
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int u = 0; u < ND; ++u) acc[u] *= inv;
      store_o<BF16, ND>(p, at, hq, lane * ND, acc);
      if (lane == 0) store_lse(p, at, hq, m, l);
    }
    if (shares > 1) __syncthreads();
  }
}

template <int D, bool BF16>
cudaError_t launch_rt(const KvAttnParams& p, int rt, int workers, int ctas, int stride, bool first, int grid,
                      cudaStream_t st) {
  auto kern = rt == 8 ? kv_join_kernel<D, 8, BF16> : rt == 16 ? kv_join_kernel<D, 16, BF16> : kv_join_kernel<D, kKvPrRows, BF16>;
  return launch_after_previous(kern, grid, kJoinWarps * 32, 0, st, p, workers, ctas, stride, first);
}

}  // namespace

cudaError_t launch_kv_join(const KvAttnParams& p, bool bf16, int rt, int workers, int ctas, int stride, bool first,
                           int grid, cudaStream_t st) {
  if (p.D == 64)
    return bf16 ? launch_rt<64, true>(p, rt, workers, ctas, stride, first, grid, st)
                : launch_rt<64, false>(p, rt, workers, ctas, stride, first, grid, st);
  return bf16 ? launch_rt<128, true>(p, rt, workers, ctas, stride, first, grid, st)
              : launch_rt<128, false>(p, rt, workers, ctas, stride, first, grid, st);
}

}  // namespace ab
