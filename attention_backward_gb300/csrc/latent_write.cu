// Rows of new tokens into the latent cache: the latent vector normalised, the
// key part turned to its position (include/attn_latent.h).
//
// Bound by HBM (1152 bytes in and out a token), by latency for few tokens.  A warp
// takes a token: two 16-byte pieces of c a lane, whose squares are summed across the
// warp, and one of the 32 pairs of k a lane.  26859 tokens, normalised and turned: 10.9 us,
// 5.7 TB/s, 84 % of the copy rate.
#include "cvt.cuh"
#include "kv_launch.h"
#include "latent.h"
#include "rope.h"
#include "sm103.cuh"

namespace ab {

namespace {

constexpr int WARPS = 4;

template <bool BF16>
__device__ __forceinline__ float one(const uint8_t* p) {
  return unpack2<BF16>(*reinterpret_cast<const uint16_t*>(p)).x;
}

template <bool BF16>
__global__ void __launch_bounds__(WARPS * 32) latent_write_kernel(const __grid_constant__ LatWriteParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int slot = p.slot_map[t];  // (its row is read meanwhile, whether it is kept or not)
  const uint8_t* const src = p.kv + 2 * t * p.kv_stride;
  uint4 x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) x[i] = *reinterpret_cast<const uint4*>(src + 16 * (lane + 32 * i));
  // my pair of k: both columns side by side, or half of them apart
  const int c1 = p.inter ? 2 * lane : lane, c2 = p.inter ? 2 * lane + 1 : lane + 32;
  const uint8_t* const k = src + 2 * kLatDim;
  float k1 = one<BF16>(k + 2 * c1), k2 = one<BF16>(k + 2 * c2);
  if (p.steps != nullptr) {
    float c, s;
    turn(p.pos[t], p.steps[lane], &c, &s);
    c *= p.scale, s *= p.scale;
    const float y = k1 * c - k2 * s;
    k2 = k1 * s + k2 * c;
    k1 = y;
  }
  if (p.weight != nullptr) {
    uint4 w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = *reinterpret_cast<const uint4*>(p.weight + 16 * (lane + 32 * i));
    uint32_t* const u = reinterpret_cast<uint32_t*>(x);
    const uint32_t* const v = reinterpret_cast<const uint32_t*>(w);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 a = unpack2<BF16>(u[i]);
      sum += a.x * a.x + a.y * a.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float r = 1.f / sqrtf(sum * (1.f / kLatDim) + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 a = unpack2<BF16>(u[i]), b = unpack2<BF16>(v[i]);
      u[i] = pack2<BF16>(a.x * r * b.x, a.y * r * b.y);
    }
  }
  const uint32_t kk = pack2<BF16>(k1, k2);
  const bool held = slot >= 0 && slot < p.slots;
  auto store = [&](uint8_t* dst) {
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<uint4*>(dst + 16 * (lane + 32 * i)) = x[i];
    dst += 2 * kLatDim;
    *reinterpret_cast<uint16_t*>(dst + 2 * c1) = static_cast<uint16_t>(kk & 0xffffu);
    *reinterpret_cast<uint16_t*>(dst + 2 * c2) = static_cast<uint16_t>(kk >> 16);
  };
  __syncwarp();  // (out may be kv: every lane has read its row)
  if (held) store(p.cache + 2 * (static_cast<int64_t>(slot) * p.row_stride));
  if (p.out != nullptr) store(p.out + 2 * t * p.out_stride);
}

}  // namespace

cudaError_t launch_latent_write(const LatWriteParams& p, bool bf16, cudaStream_t st) {
  const unsigned blocks = static_cast<unsigned>((p.T + WARPS - 1) / WARPS);
  return launch_chained(bf16 ? latent_write_kernel<true> : latent_write_kernel<false>, dim3(blocks), WARPS * 32, 0, st,
                        p);
}

}  // namespace ab
