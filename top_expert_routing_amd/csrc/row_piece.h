// Eight neighbouring values of a row of bf16 or fp32, as fp32.
#pragma once

#include "common.h"

namespace moe {

struct Piece {
  float v[8];
};

template <bool BF16>
__device__ __forceinline__ Piece load8(const void* x, size_t i) {
  Piece p;
  if constexpr (BF16) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      p.v[2 * j] = __uint_as_float(w[j] << 16);
      p.v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + i + 4);
    p = Piece{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  }
  return p;
}

// The same in two steps, so that many pieces are asked for before the first is waited for.
struct RawPiece {
  uint4 u[2];              // bf16: the first only
};
__device__ __forceinline__ RawPiece load8_raw(bool bf16, const void* x, size_t i) {
  RawPiece r;
  if (bf16) {
    r.u[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i);
    r.u[1] = r.u[0];
  } else {
    r.u[0] = *reinterpret_cast<const uint4*>(static_cast<const float*>(x) + i);
    r.u[1] = *reinterpret_cast<const uint4*>(static_cast<const float*>(x) + i + 4);
  }
  return r;
}
__device__ __forceinline__ Piece unpack8(bool bf16, const RawPiece& r) {
  const uint32_t w[8] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w, r.u[1].x, r.u[1].y, r.u[1].z, r.u[1].w};
  Piece p;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    p.v[j] = __uint_as_float(bf16 ? (j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16) : w[j]);
  return p;
}

__device__ __forceinline__ void store8(bool bf16, void* y, size_t i, const Piece& p) {
  if (bf16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + i) =
        make_uint4(pack_bf16x2(p.v[0], p.v[1]), pack_bf16x2(p.v[2], p.v[3]), pack_bf16x2(p.v[4], p.v[5]),
                   pack_bf16x2(p.v[6], p.v[7]));
  } else {
    float* o = static_cast<float*>(y) + i;
    *reinterpret_cast<float4*>(o) = make_float4(p.v[0], p.v[1], p.v[2], p.v[3]);
    *reinterpret_cast<float4*>(o + 4) = make_float4(p.v[4], p.v[5], p.v[6], p.v[7]);
  }
}

}  // namespace moe
