// Row quantiser (moe_quantize_rows_i8, and the token rows of moe_grouped_ffn_i8).
//
// One pass: a row's values are loaded once, all loads of a lane in flight
// together, stay in registers through the maximum, and leave as codes.  Bound by
// memory: 3 (bf16) or 5 (fp32) bytes a value.  A block of four wavefronts takes a row,
// or, where a row has no more values than the loads of one wavefront, each
// wavefront one.  (A wavefront per row at every size: bf16 4096 x 2048 9.8 us against 8.1,
// 8192 x 2880 21.2 us against 17.5, which is 4.04 TB/s; a row's loads and roundings are
// one chain.)  Rows of more than 256 * 8 * kMaxHeld values are read twice.
#include "launch.h"
#include "quantize.h"
#include "row_piece.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxHeld = 8;     // 8-value pieces of a row a lane holds

__device__ __forceinline__ uint32_t piece_max(const Piece& p) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, abs_bits(p.v[j]));
  return m;
}

// LANES threads per row; HELD pieces each (0: the row is read again for its codes).
template <bool BF16, int LANES, int HELD>
__global__ __launch_bounds__(kThreads) void quantize_rows(const void* __restrict__ x, int T, int d,
                                                          int8_t* __restrict__ q, float* __restrict__ s) {
  __shared__ uint32_t part[kThreads / kWave];
  const int t = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES, l = threadIdx.x % LANES;
  if (LANES == kWave && t >= T) return;         // one row per block otherwise
  const size_t row = static_cast<size_t>(t) * d;
  Piece held[HELD > 0 ? HELD : 1];
  uint32_t m = 0;
  if constexpr (HELD > 0) {
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      const int i = (h * LANES + l) * 8;
      if (i < d) held[h] = load8<BF16>(x, row + i);
    }
#pragma unroll
    for (int h = 0; h < HELD; ++h)
      if ((h * LANES + l) * 8 < d) m = max(m, piece_max(held[h]));
  } else {
    // unsigned: the last step of a row next to 2^31 values passes int32
    for (uint32_t i = l * 8; i < static_cast<uint32_t>(d); i += LANES * 8) m = max(m, piece_max(load8<BF16>(x, row + i)));
  }
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o, kWave)));
  if constexpr (LANES > kWave) {
    if (lane_id() == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < LANES / kWave; ++w) m = max(m, part[w]);
  }
  const QuantScale qs = quant_scale(m);
  if constexpr (HELD > 0) {
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      const int i = (h * LANES + l) * 8;
      if (i < d) *reinterpret_cast<uint2*>(q + row + i) = quant_codes8(held[h].v, qs);
    }
  } else {
    for (uint32_t i = l * 8; i < static_cast<uint32_t>(d); i += LANES * 8)
      *reinterpret_cast<uint2*>(q + row + i) = quant_codes8(load8<BF16>(x, row + i).v, qs);
  }
  if (l == 0) s[t] = qs.scale;
}

template <bool BF16>
void launch_rows(const void* x, int T, int d, int8_t* q, float* s, hipStream_t stream) {
  dim3 block(kThreads);
  if (d <= kWave * 8) {
    const dim3 grid((T + kThreads / kWave - 1) / (kThreads / kWave));
    hipLaunchKernelGGL((quantize_rows<BF16, kWave, 1>), grid, block, 0, stream, x, T, d, q, s);
    return;
  }
  const int pieces = (d / 8 + kThreads - 1) / kThreads;
  const dim3 grid(T);
  if (pieces <= 1) hipLaunchKernelGGL((quantize_rows<BF16, kThreads, 1>), grid, block, 0, stream, x, T, d, q, s);
  else if (pieces <= 2) hipLaunchKernelGGL((quantize_rows<BF16, kThreads, 2>), grid, block, 0, stream, x, T, d, q, s);
  else if (pieces <= 4) hipLaunchKernelGGL((quantize_rows<BF16, kThreads, 4>), grid, block, 0, stream, x, T, d, q, s);
  else if (pieces <= kMaxHeld) hipLaunchKernelGGL((quantize_rows<BF16, kThreads, kMaxHeld>), grid, block, 0, stream, x, T, d, q, s);
  else hipLaunchKernelGGL((quantize_rows<BF16, kThreads, 0>), grid, block, 0, stream, x, T, d, q, s);
}

}  // namespace

hipError_t launch_quantize_rows(const void* x, int bf16, int T, int d, int8_t* q, float* s, hipStream_t stream) {
  // a grid has fewer than 2^32 threads: at most 2^23 rows of a block each in a launch
  constexpr int kMost = 1 << 23;
  for (int t = 0; t < T; t += kMost) {
    const int n = T - t < kMost ? T - t : kMost;
    const size_t at = static_cast<size_t>(t) * d;
    const void* xt = static_cast<const char*>(x) + at * (bf16 ? 2 : 4);
    if (bf16) launch_rows<true>(xt, n, d, q + at, s + t, stream);
    else launch_rows<false>(xt, n, d, q + at, s + t, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (n < kMost) break;                       // t + kMost may pass int32
  }
  return hipSuccess;
}

}  // namespace moe
