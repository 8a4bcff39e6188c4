// int8 quantisation shared by the row quantiser and the FFN's epilogue:
//   scale = max |v| * fl(1 / 127) in fp32 (1 where that is 0; NaN unless all v are finite)
//   code  = RNE(v / scale), the quotient exact, held to [-127, 127].
#pragma once

#include "common.h"

namespace moe {

// Running maximum of magnitudes as bit patterns: infinities and NaNs are above
// every finite magnitude, so one of them survives to the scale.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct QuantScale {
  float scale;   // what is stored
  float s, r;    // divisor of the codes (times `up`), about its reciprocal
  float up;      // 2^64 for scales near the subnormals, where r would overflow; exact either way
};

__device__ __forceinline__ QuantScale quant_scale(uint32_t amax_bits) {
  QuantScale q;
  const float amax = __uint_as_float(amax_bits);
  const bool finite = amax_bits < 0x7f800000u;
  float s = amax * (1.0f / 127.0f);
  if (s == 0.0f) s = 1.0f;
  q.up = s < 0x1p-90f ? 0x1p64f : 1.0f;
  q.scale = finite ? s : __builtin_nanf("");
  q.s = finite ? s * q.up : 1.0f;
  q.r = finite ? __builtin_amdgcn_rcpf(q.s) : 0.0f;
  return q;
}

// The code of v: v * r is within a few ulp of the quotient, so its nearest
// integer c is the right one or, next to a half, its neighbour.  The remainder
// v - c * s (one fma; exact wherever it decides) tells: past half a step the
// neighbour is nearer, at exactly half a step the even one is taken.
__device__ __forceinline__ int quant_code(float v, const QuantScale& q) {
  const float x = v * q.up;
  float c = rintf(x * q.r);
  const float e = __builtin_fmaf(-c, q.s, x);
  const float h = 0.5f * q.s, m = fabsf(e);
  const int ci = static_cast<int>(c);
  if (m > h || (m == h && (ci & 1))) c += __builtin_copysignf(1.0f, e);
  c = fminf(fmaxf(c, -127.0f), 127.0f);
  return q.r == 0.0f ? 0 : static_cast<int>(c);
}

__device__ __forceinline__ uint32_t pack_codes(int a, int b, int c, int d) {
  return (a & 0xff) | ((b & 0xff) << 8) | ((c & 0xff) << 16) | (static_cast<uint32_t>(d) << 24);
}

}  // namespace moe
