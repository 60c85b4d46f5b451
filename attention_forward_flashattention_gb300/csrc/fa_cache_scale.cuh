// Scales of the block cache, powers of two, and codes brought from one to another.
#pragma once

#include "ptx.cuh"

namespace fa {

// The smallest power of two that is not below x (a positive normal number).
__device__ __forceinline__ float pow2_above(float x) {
  const uint32_t u = __float_as_uint(x);
  return __uint_as_float((u + 0x7FFFFFu) & 0xFF800000u);
}

// Four codes times f, rounded to codes again.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float f) {
  const float2 lo = ptx::e4m3x2_to_f32(c & 0xFFFFu), hi = ptx::e4m3x2_to_f32(c >> 16);
  return ptx::pack4_e4m3(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
}
__device__ __forceinline__ uint4 rescale16(uint4 u, float f) {
  return make_uint4(rescale4(u.x, f), rescale4(u.y, f), rescale4(u.z, f), rescale4(u.w, f));
}

}  // namespace fa
