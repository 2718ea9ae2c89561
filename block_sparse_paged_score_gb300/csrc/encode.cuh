// encode.cuh -- the rule both cache writers quantise MXFP4 groups by.
#pragma once

#include <stdint.h>

namespace bsp {

// Shared exponent of an MXFP4 group: clamp(floor(log2(amax)) - 2, -127, 127),
// floor(log2) read exactly off the fp32 bits (OCP MX v1.0 rule).
__device__ __forceinline__ int mx_shared_exp(float amax) {
  uint32_t b = __float_as_uint(amax);
  if (b == 0) return -127;
  int ex = (b >> 23) & 0xFF;
  int E = ex ? ex - 127 : (31 - __clz(b & 0x7FFFFFu)) - 149;
  int e = E - 2;
  return e < -127 ? -127 : (e > 127 ? 127 : e);
}

}  // namespace bsp
