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

// The low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x0c0c0400u);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// The codes of eight values of one row (its scale the same for the whole wavefront).
// Adding 1.5 * 2^23 to v * r rounds it to the nearest integer c and leaves c's two's
// complement in the low bits.  c is right if the remainder stays below half a step;
// where some lane's does not (next to a border, 1 of 10^5 values), or the scale is
// not an ordinary one, the wavefront takes quant_code.
__device__ __forceinline__ uint2 quant_codes8(const float (&v)[8], const QuantScale& q) {
  constexpr float kMagic = 12582912.0f;
  uint32_t c[8];
  float far = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float m = __builtin_fmaf(v[j], q.r, kMagic);
    c[j] = __float_as_uint(m);
    far = fmaxf(far, fabsf(__builtin_fmaf(kMagic - m, q.s, v[j])));
  }
  const bool plain = q.up == 1.0f && q.r != 0.0f && far < 0.5f * q.s;
  if (__all(plain)) return make_uint2(low_bytes(c[0], c[1], c[2], c[3]), low_bytes(c[4], c[5], c[6], c[7]));
  int e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] = quant_code(v[j], q);
  return make_uint2(pack_codes(e[0], e[1], e[2], e[3]), pack_codes(e[4], e[5], e[6], e[7]));
}

}  // namespace moe
