// The 8-bit checkpoint format on the device (include/rcu.h describes it).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rcu.h"

namespace rcu {

__device__ __forceinline__ float power2(int e) { return __int_as_float((e + 127) << 23); }

// The smallest e in [-126, 121] with top <= 127 * 2^e (top >= 0, finite).
// top = m * 2^k with m in [1, 2): 127 * 2^e reaches it for e = k - 6 exactly
// when m * 64 <= 127, that is when the fraction is at most 63/64.  At e = 122
// a code of 64 would already stand for infinity, so e stops at 121 and the
// codes of a larger top at 127.
__device__ __forceinline__ int act8_exponent(float top) {
  const int bits = __float_as_int(top);
  const int e = (bits >> 23) - 127 - 6 + ((bits & 0x7fffff) > 0x7e0000);
  return min(max(e, -126), 121);
}

// The code of v at the scale inv = 2^-e: rounded to the nearest even, -128 for
// what is not finite.
__device__ __forceinline__ int act8_code(float v, float inv) {
  return isfinite(v) ? min(max(__float2int_rn(v * inv), -127), 127) : -128;
}

// What a code stands for.
__device__ __forceinline__ float act8_value(int code, int e) {
  return code == -128 ? __int_as_float(0x7fc00000) : (float)code * power2(e);
}

// Four codes of one word as fp32 whole numbers: c + 128 in the low byte of 2^23
// is exact.  Code -128 comes out as -128 here; act8_any_nan tells whether a word
// holds one (a byte of w ^ 0x80808080 is 0 then).
__device__ __forceinline__ float act8_whole(uint32_t w, int j) {
  return __uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4b000000u, 0x7540 + j)) - 8388736.f;
}
__device__ __forceinline__ bool act8_any_nan(uint32_t w) {
  const uint32_t t = w ^ 0x80808080u;
  return ((t - 0x01010101u) & ~t & 0x80808080u) != 0;
}

}  // namespace rcu
