// Rotary positions of queries and keys in one launch, in place or into other
// tensors; its inverse is the gradient (include/attn_rope.h).
//
// Bound by HBM: 2 bytes in and 2 out a value.  A thread owns 8 pairs of one
// token, 16 columns in two 16-byte pieces in either layout, makes their cos and
// sin once and turns them in several heads, STEP heads in flight.
#include "cvt.cuh"
#include "kv_launch.h"
#include "rope.h"
#include "sm103.cuh"

namespace ab {

namespace {

constexpr int THREADS = 128, STEP = 4;

template <bool BF16, bool INTER>
__device__ __forceinline__ void turn_pairs(uint4* a, uint4* b, const float* c, const float* s) {
  uint32_t* const u = reinterpret_cast<uint32_t*>(a);
  uint32_t* const v = reinterpret_cast<uint32_t*>(b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTER) {  // u, v: pairs 0-3 and 4-7 side by side
      const float2 x = unpack2<BF16>(u[i]), z = unpack2<BF16>(v[i]);
      u[i] = pack2<BF16>(x.x * c[i] - x.y * s[i], x.x * s[i] + x.y * c[i]);
      v[i] = pack2<BF16>(z.x * c[i + 4] - z.y * s[i + 4], z.x * s[i + 4] + z.y * c[i + 4]);
    } else {  // u: the first columns of the 8 pairs, v: the second
      const float2 x = unpack2<BF16>(u[i]), z = unpack2<BF16>(v[i]);
      const float* const cc = c + 2 * i;
      const float* const ss = s + 2 * i;
      u[i] = pack2<BF16>(x.x * cc[0] - z.x * ss[0], x.y * cc[1] - z.y * ss[1]);
      v[i] = pack2<BF16>(x.x * ss[0] + z.x * cc[0], x.y * ss[1] + z.y * cc[1]);
    }
  }
}

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(THREADS) rope_kernel(const __grid_constant__ RopeParams p) {
  grid_dependents_launch();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x;
  const int64_t token = id / p.lanes;
  const int lane = static_cast<int>(id - token * p.lanes);
  const int h0 = lane / p.per_head, j = lane % p.per_head;
  const int b = static_cast<int>(token / p.S), t = static_cast<int>(token % p.S);
  const bool live = b < p.B, turns = j < p.R / 16;
  float c[8], s[8];
  if (live && turns) {  // (positions and steps may come from the launch before)
    grid_dependency_wait();
    const int pos = p.pos[b * p.pos_b + t];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      turn(pos, p.steps[j * 8 + i], &c[i], &s[i]);
      c[i] *= p.scale, s[i] *= p.inverse ? -p.scale : p.scale;
    }
  } else {
    grid_dependency_wait();
  }
  if (!live) return;
  const int first = turns ? (INTER ? 16 * j : 8 * j) : 0, gap = INTER ? 8 : p.R / 2;
  for (int h = h0; h < p.heads; h += STEP * p.stride) {
    uint4 x[STEP][2];
    uint8_t* to[STEP][2];
#pragma unroll
    for (int k = 0; k < STEP; ++k) {
      to[k][0] = to[k][1] = nullptr;
      int hh = h + k * p.stride;
      if (hh >= p.heads) continue;
      const bool other = hh >= p.t[0].H;
      const RopeTensor& r = p.t[other];
      hh -= other ? p.t[0].H : 0;
      int at[2] = {r.start + first, r.start + first + gap};
      bool on[2] = {true, true};
      if (!turns) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // pieces before the rotated columns, then behind them
          const int piece = 2 * (j - p.R / 16) + e;
          on[e] = piece < r.copies;
          at[e] = 8 * piece < r.start ? 8 * piece : 8 * piece + p.R;
        }
      }
      const uint8_t* const from = r.x + 2 * (b * r.sx_b + t * r.sx_s + hh * r.sx_h);
      uint8_t* const dst = r.y + 2 * (b * r.sy_b + t * r.sy_s + hh * r.sy_h);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (on[e]) {
          x[k][e] = *reinterpret_cast<const uint4*>(from + 2 * at[e]);
          to[k][e] = dst + 2 * at[e];
        }
    }
#pragma unroll
    for (int k = 0; k < STEP; ++k) {
      if (turns && to[k][0]) turn_pairs<BF16, INTER>(&x[k][0], &x[k][1], c, s);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (to[k][e]) *reinterpret_cast<uint4*>(to[k][e]) = x[k][e];
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p0, bool bf16, int sms, cudaStream_t st) {
  RopeParams p = p0;
  const int64_t tokens = static_cast<int64_t>(p.B) * p.S;
  const int copies = p.t[0].copies > p.t[1].copies ? p.t[0].copies : p.t[1].copies;
  p.per_head = p.R / 16 + (copies + 1) / 2;
  // Heads a thread: as many as leave a full machine (2048 threads an SM), at most 8.
  int each = 1;
  while (each < 8 && each < p.heads && tokens * p.per_head * ((p.heads + 2 * each - 1) / (2 * each)) >= int64_t(sms) * 2048)
    each *= 2;
  p.stride = (p.heads + each - 1) / each;
  p.lanes = p.per_head * p.stride;
  const int64_t blocks = (tokens * p.lanes + THREADS - 1) / THREADS;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  auto kern = bf16 ? (p.inter ? rope_kernel<true, true> : rope_kernel<true, false>)
                   : (p.inter ? rope_kernel<false, true> : rope_kernel<false, false>);
  return launch_chained(kern, dim3(static_cast<unsigned>(blocks)), THREADS, 0, st, p);
}

}  // namespace ab
