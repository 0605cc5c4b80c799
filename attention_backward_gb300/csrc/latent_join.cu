// The second launch of attention over latent rows: rows whose keys were split over
// CTAs are joined from their f32 partials in the workspace, in a fixed order.
//
// Lists: each unit is lp.splits parts in as many slots.  The cache:
// entry w of ``desc`` (first token of the request, first row of the unit in the
// request, rows, first part) names the unit that CTA w finished and did not begin; its
// parts are d.w to w / group in order, w = -1 where there is none.  Each half of a row
// of such a unit is an item; a warp takes one, or, where there are warps to spare, 2 to
// 16 of a block take fixed shares of its parts.  Four parts are in flight, the first while
// the weights are made: latency-bound, 5 to 8 us, of which 27 MB of parts (64 requests of 64
// heads on 152 CTAs) take 5.
#include "cvt.cuh"
#include "kv_launch.h"
#include "latent.h"
#include "sm103.cuh"

namespace ab {

namespace {

constexpr int WARPS = 16, HALF = kLatDim / 2, ND = HALF / 32, PF = 4;  // columns of an item and of a lane, parts in flight
constexpr int LISTERS = (kLatMaxCtas + 31) / 32;  // warps that hold entries, one a thread
static_assert(LISTERS <= WARPS, "an entry a thread");

template <bool LISTS, bool BF16>
__global__ void __launch_bounds__(WARPS * 32, 2) latent_join_kernel(const __grid_constant__ LatParams lp, int group, int ctas) {
  const KvAttnParams& p = lp.a;
  __shared__ int4 list[kLatMaxCtas];
  __shared__ int counts[WARPS];
  __shared__ float s_o[WARPS][HALF];
  __shared__ float2 s_ml[WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  int count = 0;
  if constexpr (LISTS) {
    count = lp.B * lp.S * lp.HKV;
  } else {
    if (blockIdx.x == 0) {  // the call's error word: some CTA's error, if there is any
      const int err = tid < ctas ? p.cta_err[tid] : kErrNone;
      if (tid == 0) *p.err = kErrNone;
      if (__syncthreads_or(err != kErrNone) && err != kErrNone) *p.err = err;
    }
    int4 d = make_int4(0, 0, 0, -1);
    if (tid < ctas) d = p.desc[tid];
    const uint32_t held = __ballot_sync(0xffffffffu, d.w >= 0);
    if (lane == 0) counts[warp] = __popc(held);
    __syncthreads();
    int first = 0;
#pragma unroll
    for (int i = 0; i < LISTERS; ++i) {
      if (i < warp) first += counts[i];
      count += counts[i];
    }
    // parts in the upper half of z, this CTA's place in its group in the upper half of w
    if (d.w >= 0)
      list[first + __popc(held & ((1u << lane) - 1u))] = make_int4(d.x, d.y, d.z | (tid / group - d.w + 1) << 16, d.w | (tid % group) << 16);
    __syncthreads();
  }
  const int items = count * kLatRows * 2;
  int ls = 0;  // log2 of the warps an item
  while ((1 << ls) < WARPS && items << (ls + 1) <= static_cast<int>(gridDim.x) * WARPS) ++ls;
  const int shares = 1 << ls, per_block = WARPS >> ls, share = warp & (shares - 1);
  for (int t0 = blockIdx.x * per_block; t0 < items; t0 += gridDim.x * per_block) {
    const int item = t0 + (warp >> ls);
    int4 u = make_int4(0, 0, 0, 0);
    if (!LISTS && item < items) u = list[item / (2 * kLatRows)];
    const int unit = item / (2 * kLatRows), row = item / 2 % kLatRows, half = item % 2;
    const int live = LISTS ? lp.gh : u.z & 0xffff, parts = LISTS ? lp.splits : u.z >> 16, g0 = u.w & 0xffff, sub = u.w >> 16;
    const bool on = item < items && row < live;
    auto slot_of = [&](int i) { return LISTS ? unit * lp.splits + i : 2 * ((g0 + i) * group + sub) + (i == 0 ? 1 : 0); };
    float m = -INFINITY, l = 0.f, acc[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) acc[i] = 0.f;
    if (on) {
      const int i1 = parts * (share + 1) >> ls;
      for (int i0 = parts * share >> ls; i0 < i1; i0 += 32) {
        const int n = imin(32, i1 - i0);
        float2 v = make_float2(0.f, 0.f);
        if (lane < n) v = p.part_ml[static_cast<int64_t>(slot_of(i0 + lane)) * kLatRows + row];
        float4 x[PF][ND / 4];
        auto load = [&](int i) {  // parts i .. i + PF - 1
#pragma unroll
          for (int k = 0; k < PF; ++k) {
            const float4* const src = reinterpret_cast<const float4*>(
                p.part_o + (static_cast<int64_t>(slot_of(i0 + imin(i + k, n - 1))) * kLatRows + row) * kLatDim + half * HALF);
#pragma unroll
            for (int e = 0; e < ND / 4; ++e) x[k][e] = src[e * 32 + lane];
          }
        };
        load(0);  // (in flight while the weights are made)
        float mx = v.y == 0.f ? -INFINITY : v.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mx = fmaxf(mx, m);
        const float w = v.y == 0.f ? 0.f : ex2((v.x - mx) * p.scale_log2), g = m == -INFINITY ? 0.f : ex2((m - mx) * p.scale_log2);
        m = mx;
        float sum = w * v.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * g + sum;
#pragma unroll
        for (int i = 0; i < ND; ++i) acc[i] *= g;
        for (int i = 0; i < n; i += PF) {
          if (i > 0) load(i);
#pragma unroll
          for (int k = 0; k < PF; ++k) {
            const float f = __shfl_sync(0xffffffffu, w, (i + k) & 31);
            if (i + k < n && f != 0.f) {  // (a part that saw no key of the row says nothing)
#pragma unroll
              for (int e = 0; e < ND / 4; ++e) {
                acc[4 * e] += f * x[k][e].x, acc[4 * e + 1] += f * x[k][e].y;
                acc[4 * e + 2] += f * x[k][e].z, acc[4 * e + 3] += f * x[k][e].w;
              }
            }
          }
        }
      }
      if (share > 0) {
#pragma unroll
        for (int i = 0; i < ND; ++i) s_o[warp][i * 32 + lane] = acc[i];
        if (lane == 0) s_ml[warp] = make_float2(m, l);
      }
    }
    if (shares > 1) __syncthreads();
    if (on && share == 0) {
      for (int k = 1; k < shares; ++k) {
        const float2 v = s_ml[warp + k];
        if (v.y == 0.f) continue;
        const float mx = fmaxf(m, v.x), g = l == 0.f ? 0.f : ex2((m - mx) * p.scale_log2), f = ex2((v.x - mx) * p.scale_log2);
        l = l * g + v.y * f;
        m = mx;
#pragma unroll
        for (int i = 0; i < ND; ++i) acc[i] = acc[i] * g + s_o[warp + k][i * 32 + lane] * f;
      }
      int64_t o_at, lse_at;
      if constexpr (LISTS) {
        const LatListUnit v = list_unit(unit, lp);
        const int head = v.g * lp.gh + row;
        o_at = v.b * lp.so_b + v.t * p.so_s + head * p.so_h, lse_at = v.b * lp.sl_b + head * p.sl_h + v.t * p.sl_s;
      } else {
        const int at = u.y + row, head = at % p.G;  // row of the request
        const int64_t t = static_cast<int64_t>(u.x) + at / p.G;
        o_at = t * p.so_s + head * p.so_h, lse_at = head * p.sl_h + t * p.sl_s;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint8_t* const out = p.o + 2 * (o_at + half * HALF);
#pragma unroll
      for (int e = 0; e < ND / 4; ++e) {
        const uint2 w = make_uint2(pack2<BF16>(acc[4 * e] * inv, acc[4 * e + 1] * inv),
                                   pack2<BF16>(acc[4 * e + 2] * inv, acc[4 * e + 3] * inv));
        *reinterpret_cast<uint2*>(out + 8 * (e * 32 + lane)) = w;
      }
      if (lane == 0 && half == 0)
        p.lse[lse_at] = l == 0.f ? -INFINITY : (fmaf(m, p.scale_log2, -kLatTop) + log2f(l)) * 0.69314718055994531f;
    }
    if (shares > 1) __syncthreads();
  }
}

}  // namespace

cudaError_t launch_latent_join(const LatParams& p, bool bf16, int group, int ctas, int sms, cudaStream_t st) {
  auto kern = group == 0 ? (bf16 ? latent_join_kernel<true, true> : latent_join_kernel<true, false>)
                         : (bf16 ? latent_join_kernel<false, true> : latent_join_kernel<false, false>);
  return launch_chained(kern, dim3(2 * sms), WARPS * 32, 0, st, p, group, ctas);
}

}  // namespace ab
