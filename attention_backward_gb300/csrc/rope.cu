// Rotary positions of queries and keys in one launch, in place or into other
// tensors; its inverse is the gradient (include/attn_rope.h).
//
// Bound by HBM: 2 bytes in and 2 out a value.  A thread owns 8 pairs of one
// token, 16 columns in two 16-byte pieces in either layout, and turns them in several
// heads, STEP heads in flight.  A block makes the cosines and sines of its tokens in
// shared memory, one or two a thread, while the first heads are on their way (eight a
// thread, and 96 registers: 14.4 us instead of 6.9 for 2048 tokens of 20 heads of 192,
// 64 of them turned).  32 and 4 heads of 128, 16384 tokens: 51 us, 5.9 TB/s, 87 % of the
// copy rate.  64 columns of 65 heads of 576, 4096 tokens: 14.8 us, 4.6 TB/s, in pieces of
// 128 bytes.
#include "cvt.cuh"
#include "kv_launch.h"
#include "rope.h"
#include "sm103.cuh"

namespace ab {

namespace {

constexpr int THREADS = 128, STEP = 2;
constexpr int PAIRS = 8 * THREADS;  // most pairs of a block's tokens: 8 a thread

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
__global__ void __launch_bounds__(THREADS, 8) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 table[PAIRS];  // (cos, sin) of the block's tokens and pairs
  grid_dependents_launch();
  const int tokens = p.B * p.S, half = p.R / 2;
  int token, lane, token0;  // mine, and the block's first
  bool live;
  if (p.split == 1) {  // several tokens a block
    const int k = static_cast<int>(threadIdx.x) / p.lanes;
    token0 = blockIdx.x * p.share, token = token0 + k, lane = threadIdx.x - k * p.lanes;
    live = k < p.share && token < tokens;
  } else {  // several blocks a token
    token = token0 = blockIdx.x / p.split, lane = (blockIdx.x - token * p.split) * p.share + threadIdx.x;
    live = static_cast<int>(threadIdx.x) < p.share && lane < p.lanes;
  }
  const int b = token / p.S, t = token - b * p.S;
  int h = lane / p.per_head;  // next head, those of k behind those of q
  const int j = lane - h * p.per_head;
  const bool turns = j < p.R / 16;
  const int heads = live ? p.heads : 0;
  // My two pieces of a head: where they begin, and whether they are there.  Threads
  // behind those that turn copy the columns before the turned ones, then those after.
  auto pieces = [&](const RopeTensor& r, int* at, bool* on) {
    at[0] = r.start + (INTER ? 16 : 8) * j, at[1] = at[0] + (INTER ? 8 : half);
    on[0] = on[1] = true;
    if (!turns) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int piece = 2 * (j - p.R / 16) + e;
        on[e] = piece < r.copies;
        at[e] = 8 * piece < r.start ? 8 * piece : 8 * piece + p.R;
      }
    }
  };
  int at[2];
  bool on[2];
  const RopeTensor* r = &p.t[0];
  int past = 0, end = p.t[0].H;  // heads before this tensor's, and up to its end
  const uint8_t* from;
  uint8_t* to;
  auto enter = [&]() {  // the tensor of head h
    if (h >= end && past == 0) r = &p.t[1], past = end, end = p.heads;
    pieces(*r, at, on);
    from = r->x + 2 * (b * r->sx_b + t * r->sx_s), to = r->y + 2 * (b * r->sy_b + t * r->sy_s);
  };
  uint4 x[STEP][2];
  auto load = [&]() {  // heads h, h + stride, .. of the tensor
#pragma unroll
    for (int k = 0; k < STEP; ++k) {
      const int hh = h + k * p.stride;
      if (hh >= end) break;
      const uint8_t* const src = from + 2 * (hh - past) * r->sx_h;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (on[e]) x[k][e] = *reinterpret_cast<const uint4*>(src + 2 * at[e]);
    }
  };
  grid_dependency_wait();  // (all inputs may come from the launch before)
  if (h < heads) {
    enter();
    load();  // in flight while the table is made
  }
  const int pairs = (p.split == 1 ? (p.share < tokens - token0 ? p.share : tokens - token0) : 1) * half;
  for (int i = threadIdx.x; i < pairs; i += THREADS) {
    const int k = i / half, n = token0 + k, row = n / p.S;
    float2 cs;
    turn(p.pos[row * p.pos_b + (n - row * p.S)], p.steps[i - k * half], &cs.x, &cs.y);
    table[i] = make_float2(cs.x * p.scale, cs.y * (p.inverse ? -p.scale : p.scale));
  }
  __syncthreads();
  float c[8], s[8];
  if (h < heads && turns) {
    const float4* const mine = reinterpret_cast<const float4*>(table + (token - token0) * half + 8 * j);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 y = mine[i];
      c[2 * i] = y.x, s[2 * i] = y.y, c[2 * i + 1] = y.z, s[2 * i + 1] = y.w;
    }
  }
  while (h < heads) {
#pragma unroll
    for (int k = 0; k < STEP; ++k) {
      const int hh = h + k * p.stride;
      if (hh >= end) break;
      if (turns) turn_pairs<BF16, INTER>(&x[k][0], &x[k][1], c, s);
      uint8_t* const dst = to + 2 * (hh - past) * r->sy_h;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (on[e]) *reinterpret_cast<uint4*>(dst + 2 * at[e]) = x[k][e];
    }
    // the next heads of this tensor, or the first ones of k
    for (int k = 0; k < STEP && h < end; ++k) h += p.stride;
    if (h >= heads) break;
    if (h >= end) enter();
    load();
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p0, bool bf16, int sms, cudaStream_t st) {
  RopeParams p = p0;
  const int64_t tokens = static_cast<int64_t>(p.B) * p.S;
  const int copies = p.t[0].copies > p.t[1].copies ? p.t[0].copies : p.t[1].copies;
  p.per_head = p.R / 16 + (copies + 1) / 2;
  // Heads a thread: as many as leave a full machine (2048 threads an SM), at most 8 (36 heads
  // of 128, 16384 tokens: 51 us, 67 with at most 4, 53 with 16).
  int each = 1;
  while (each < 8 && each < p.heads && tokens * p.per_head * ((p.heads + 2 * each - 1) / (2 * each)) >= int64_t(sms) * 2048)
    each *= 2;
  p.stride = (p.heads + each - 1) / each;
  // Where they are more than a full machine: whole blocks a token (4096 tokens of 65 heads of
  // 64 columns: 15.7 us, 20.0 with blocks of 66 threads).
  if (p.per_head * p.stride > THREADS && tokens * p.per_head * p.stride >= int64_t(sms) * 2048)
    p.stride = p.per_head * p.stride / THREADS * THREADS / p.per_head;
  p.lanes = p.per_head * p.stride;
  p.split = (p.lanes + THREADS - 1) / THREADS;
  p.share = p.split == 1 ? THREADS / p.lanes : (p.lanes + p.split - 1) / p.split;
  const int64_t blocks = p.split == 1 ? (tokens + p.share - 1) / p.share : tokens * p.split;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  auto kern = bf16 ? (p.inter ? rope_kernel<true, true> : rope_kernel<true, false>)
                   : (p.inter ? rope_kernel<false, true> : rope_kernel<false, false>);
  return launch_chained(kern, dim3(static_cast<unsigned>(blocks)), THREADS, 0, st, p);
}

}  // namespace ab
