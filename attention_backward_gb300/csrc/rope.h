// Parameter blocks, launchers and device helpers of rotary positions (internal
// to the library).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_rope.h"

namespace ab {

struct RopeTensor {
  const uint8_t* x;
  int64_t sx_b, sx_s, sx_h;  // element strides
  uint8_t* y;
  int64_t sy_b, sy_s, sy_h;
  int H, start;
  int copies;  // 16-byte pieces a head outside the rotated columns that are copied (0 in place)
};

struct RopeParams {
  RopeTensor t[2];
  int heads;  // of both tensors
  int B, S, R;
  const int* pos;
  int64_t pos_b;
  const uint64_t* steps;
  float scale;
  int inter, inverse;
  int per_head;  // threads a head: 16 rotated columns each, then 16 copied ones
  int lanes;     // threads a token: per_head * (heads / heads a thread, rounded up)
  int stride;    // heads between the heads of a thread
  int split;     // blocks a token
  int share;     // split 1: tokens a block, else a token's threads a block
};

cudaError_t launch_rope(const RopeParams& p, bool bf16, int sms, cudaStream_t st);

// cos and sin of p turns of step / 2^64.  The 64-bit product keeps the fraction of a
// turn exactly (whole turns overflow).  Its upper half is taken as a signed number of half
// turns in f32, whose 24 bits put the angle within 2^-26 turns = 9.4e-8 radians.
__device__ __forceinline__ void turn(int p, uint64_t step, float* c, float* s) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(p)) * step;
  sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f, s, c);
}

}  // namespace ab
