// Row quantiser (moe_quantize_rows_i8, and the token rows of moe_grouped_ffn_i8):
// one wavefront per row.
#include "launch.h"
#include "quantize.h"

namespace moe {

namespace {

constexpr int kWavesPerBlock = 4;

template <bool BF16>
__device__ __forceinline__ void load8(const void* x, size_t i, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i);
    const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(p[j] << 16);
      v[2 * j + 1] = __uint_as_float(p[j] & 0xffff0000u);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + i + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

// The row is read twice (the second time from the caches).
template <bool BF16>
__global__ __launch_bounds__(kWave * kWavesPerBlock) void quantize_rows(const void* __restrict__ x, int T, int d,
                                                                        int8_t* __restrict__ q, float* __restrict__ s) {
  const int t = blockIdx.x * kWavesPerBlock + (threadIdx.x >> 6), lane = lane_id();
  if (t >= T) return;
  const size_t row = static_cast<size_t>(t) * d;
  uint32_t m = 0;
  for (int i = lane * 8; i < d; i += kWave * 8) {
    float v[8];
    load8<BF16>(x, row + i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
  }
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o, kWave)));
  const QuantScale qs = quant_scale(m);
  for (int i = lane * 8; i < d; i += kWave * 8) {
    float v[8];
    int c[8];
    load8<BF16>(x, row + i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = quant_code(v[j], qs);
    *reinterpret_cast<uint2*>(q + row + i) = make_uint2(pack_codes(c[0], c[1], c[2], c[3]), pack_codes(c[4], c[5], c[6], c[7]));
  }
  if (lane == 0) s[t] = qs.scale;
}

}  // namespace

hipError_t launch_quantize_rows(const void* x, int bf16, int T, int d, int8_t* q, float* s, hipStream_t stream) {
  dim3 grid((T + kWavesPerBlock - 1) / kWavesPerBlock), block(kWave * kWavesPerBlock);
  if (bf16)
    hipLaunchKernelGGL(quantize_rows<true>, grid, block, 0, stream, x, T, d, q, s);
  else
    hipLaunchKernelGGL(quantize_rows<false>, grid, block, 0, stream, x, T, d, q, s);
  return hipGetLastError();
}

}  // namespace moe
