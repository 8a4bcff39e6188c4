// E4M3 codes with one scale per 128 values, shared by the norm, the quantiser and the products:
//   scale = max |v| * fl(1 / 448) in fp32 (1 where that is below 2^-100; NaN unless all v are finite)
//   code  = RNE to E4M3 of v / scale.
// (448 is the largest E4M3 value: quotients reach 448 * (1 + 2^-23), which rounds to it.)
#pragma once

#include "quantize.h"

namespace moe {

constexpr int kFp8Block = 128;

struct Fp8Scale {
  float base;    // divisor of the codes, and what is stored (times what the caller has left out of v)
  float r;       // 1 / (base * up), correctly rounded; 0 for values that are not all finite
  float up = 1.f;   // 2^64 for scales near the smallest (fp8_quotient)
};

__device__ __forceinline__ Fp8Scale fp8_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return Fp8Scale{__builtin_nanf(""), 0.f};
  const float s = __uint_as_float(amax_bits) * (1.0f / 448.0f);
  if (s < 0x1p-100f) return Fp8Scale{1.f, 1.f};
  const float up = s < 0x1p-90f ? 0x1p64f : 1.f;
  return Fp8Scale{s, 1.0f / (s * up), up};
}

// Four codes in a word, of quotients already taken.
__device__ __forceinline__ uint32_t fp8_codes4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return static_cast<uint32_t>(w);
}

// fl(v / base) from the correctly rounded reciprocal: v * r is within an ulp of the quotient, and
// one step with the exact remainder rounds it correctly (Markstein).  The remainder is a multiple of 2^(e - 46), e the
// sum of the exponents of q and base, and exact while that is at least 2^-149.  Quotients that are not a zero code are
// 2^-10 or more, so bases from 2^-90 on keep it exact; smaller ones are multiplied by 2^64 with their values, which
// changes no quotient.
__device__ __forceinline__ float fp8_quotient(float v, const Fp8Scale& s) {
  const float x = v * s.up, q = x * s.r;
  return __builtin_fmaf(__builtin_fmaf(-q, s.base * s.up, x), s.r, q);
}

__device__ __forceinline__ uint2 fp8_codes8(const float (&v)[8], const Fp8Scale& s) {
  if (s.r == 0.f) return make_uint2(0, 0);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = fp8_quotient(v[i], s);
  return make_uint2(fp8_codes4(q[0], q[1], q[2], q[3]), fp8_codes4(q[4], q[5], q[6], q[7]));
}

// Maximum over each 16 lanes (a DPP row); every lane takes part.
__device__ __forceinline__ uint32_t row16_max(uint32_t m) {
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x128, 0xf, 0xf, false)));
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x124, 0xf, 0xf, false)));
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x122, 0xf, 0xf, false)));
  return max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x121, 0xf, 0xf, false)));
}

}  // namespace moe
