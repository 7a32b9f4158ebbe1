// Device helpers of the 8-bit layer: E4M3 conversions and the scale of a block.
#pragma once

#include "fp8.h"
#include "train_common.cuh"

namespace ftmoe {

// Four E4M3 codes, the first in the low byte (round to nearest even, saturating; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)hi << 16 | lo;
}

// A block's scale and what its values are multiplied by, from the bits of its
// largest magnitude (as an integer, so that NaN counts as the largest and
// spoils the block).  The scale is rounded once; so is the multiplier, whose
// rounding moves a value by 2^-24 of it before the code's rounding, 2^-4.
struct BlockScale {
  float scale, mul;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
  const float a = __uint_as_float(amax_bits);
  if (a < kFp8Tiny) return {0.f, 0.f};
  return {__fdiv_rn(a, kFp8Max), __fdiv_rn(kFp8Max, a)};
}

// The larger magnitude; NaN if one is.
__device__ __forceinline__ float max_magnitude(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Rows that a call handles: `used` (a count on the device) where it is given.
// A count out of range marks the status word and is held to the range.
__device__ __forceinline__ int used_rows(const int32_t* used, int rows, uint32_t* status) {
  if (!used) return rows;
  const int n = *used;
  if (n >= 0 && n <= rows) return n;
  if (threadIdx.x == 0) set_status(status, kStatusRange);
  return n < 0 ? 0 : rows;
}

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

// The same with the approximate reciprocal at a third of the instructions: within 6 2^-24 (expf 2, the sum 1, the
// reciprocal 2, the product 1), and exp's own steps of 2^-149 where that is more.  From exp(-|z|) the reciprocal's
// argument is 1 to 2: that of 1 + exp(-z) would be flushed to zero for z < -87.3 (131072 x 640 to codes 74.6 us so,
// 79.5 us here; the sum scaled by 2^-32 86 us).
__device__ __forceinline__ float sigmoid_rcp(float z) {
  const float t = expf(-fabsf(z));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + t));
  if (z < 0.f) r *= t;
  return r;
}

}  // namespace ftmoe
