// Root-mean-square norm of rows with the residual's addition in front of it and codes behind it
// (moe_rmsnorm), and the quantiser to E4M3 codes (moe_quantize_blocks_fp8).
//
// The norm of a row r multiplies all of it by one number, rstd, so codes do not depend on it: they are
// those of p = r * w, and rstd only multiplies their scale.  So one pass over the row in registers yields
// the sum of squares and every maximum, and one exchange between the wavefronts joins them.
// Bound by memory: x, residual, residual, y and codes are 2 + 2 + 2 + 2 + 1 bytes a value in bf16.  8191 x 2880 so:
// 43.5 us (4.9 TB/s, as a copy runs); 4159 x 2048 with an fp32 residual and int8 codes alone 16.5 us.
// A row has as few wavefronts as hold it with one piece a lane, one, two or four of them, and from 257 pieces on four with as
// many pieces a lane as hold it (2, 4 or kMaxHeld); longer ones are read twice.  us of 23.6 million values, bf16 with a residual, y
// and E4M3 codes, and of 16 rows: 512 columns one wavefront 41.3 / 3.2, two 46.4 / 3.4; 1024 two 41.2 / 3.4, four 46.1 /
// 3.3; 2048 four with a piece each 40.3 / 3.3, with two 40.8 / 3.6; 2880 four with two 44.4 / 4.0, two with three 47.2 / 4.7, four
// with four 47.4 / 4.5; 6144 four with four 46.5 / 5.0, with eight 51.6 / 5.9; 16384 with eight 49.7 / 8.4, read twice 55.0 / 10.0.
#include "fp8_block.h"
#include "launch.h"
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

enum Kind { kNone, kBf16, kF32 };

// X: x's type, R: the residual's.  LANES threads per row; HELD pieces each (0: the row is read again for
// its outputs).
template <Kind X, Kind R, int LANES, int HELD>
__global__ __launch_bounds__(kThreads) void rmsnorm(NormArgs a) {
  constexpr int WAVES = LANES / kWave, ROWS = kThreads / LANES;
  __shared__ float sums[kThreads / kWave];
  __shared__ uint32_t tops[kThreads / kWave];
  const int t = blockIdx.x * ROWS + threadIdx.x / LANES, l = threadIdx.x % LANES;
  const bool there = ROWS == 1 || t < a.T;
  if (WAVES == 1 && !there) return;             // rows of several wavefronts meet at a barrier
  const int d = there ? a.d : 0, nb = (d + kFp8Block - 1) / kFp8Block;
  const size_t row = static_cast<size_t>(t) * d;

  // r of a piece at column i: the sum as it is stored
  auto add = [&](Piece& p, const Piece& r, uint32_t i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) p.v[j] += r.v[j];
    if constexpr (R == kBf16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) p.v[j] = bf16_to_f32(f32_to_bf16(p.v[j]));
    }
    store8(R == kBf16, a.residual_out, row + i, p);
  };
  auto weigh = [&](Piece& p, const Piece& w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) p.v[j] *= w.v[j];
  };
  auto squares = [&](const Piece& p) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = __builtin_fmaf(p.v[j], p.v[j], s);
    return s;
  };

  Piece held[HELD > 0 ? HELD : 1];              // p = r * w
  float sum = 0.f;
  uint32_t top = 0;
  if constexpr (HELD > 0) {
    // all of the row is asked for before the first sum is stored
    RawPiece x[HELD], r[R != kNone ? HELD : 1], w[HELD];
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      const int i = (h * LANES + l) * 8;
      if (i < d) {
        x[h] = load8_raw(X == kBf16, a.x, row + i);
        if constexpr (R != kNone) r[h] = load8_raw(R == kBf16, a.residual, row + i);
        w[h] = load8_raw(a.weight_bf16, a.weight, i);
      }
    }
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      const int i = (h * LANES + l) * 8;
      held[h] = Piece{};
      if (i < d) {
        held[h] = unpack8(X == kBf16, x[h]);
        if constexpr (R != kNone) add(held[h], unpack8(R == kBf16, r[h]), i);
        sum += squares(held[h]);
        weigh(held[h], a.weight_bf16 ? unpack8(true, w[h]) : unpack8(false, w[h]));
      }
      if (a.code == kCodeI8) top = max(top, piece_max(held[h]));
    }
  } else {
    // unsigned: the last step of a row next to 2^31 values passes int32
    for (uint32_t i = l * 8; i < static_cast<uint32_t>(d); i += LANES * 8) {
      Piece p = load8<X == kBf16>(a.x, row + i);
      if constexpr (R != kNone) add(p, load8<R == kBf16>(a.residual, row + i), i);
      sum += squares(p);
      if (a.code == kCodeI8) {
        weigh(p, unpack8(a.weight_bf16, load8_raw(a.weight_bf16, a.weight, i)));
        top = max(top, piece_max(p));
      }
    }
  }
  sum = wave_sum(sum);
  if (a.code == kCodeI8) {
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), o, kWave)));
  }
  if constexpr (WAVES > 1) {
    if (lane_id() == 0) {
      sums[threadIdx.x >> 6] = sum;
      tops[threadIdx.x >> 6] = top;
    }
    __syncthreads();
    const int w0 = threadIdx.x / LANES * WAVES;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      sum += sums[w0 + w];
      top = max(top, tops[w0 + w]);
    }
    if (!there) return;
  }
  // a row that is not finite, or whose sum of squares is not: NaN everywhere
  const float mean = sum / static_cast<float>(d);
  const float rstd = __builtin_isfinite(sum) ? 1.0f / __builtin_sqrtf(mean + a.eps) : __builtin_nanf("");
  const QuantScale qs = quant_scale(top);

  auto finish = [&](const Piece& p, int i, bool in) {          // every lane of the 16 that share a block takes part
    if (a.y && in) {
      Piece y;
#pragma unroll
      for (int j = 0; j < 8; ++j) y.v[j] = p.v[j] * rstd;
      store8(a.y_bf16, a.y, row + i, y);
    }
    if (a.code == kCodeFp8) {
      const Fp8Scale fs = fp8_scale(row16_max(piece_max(p)));
      if (in) *reinterpret_cast<uint2*>(a.q + row + i) = fp8_codes8(p.v, fs);
      if (in && i % kFp8Block == 0) a.s[static_cast<size_t>(t) * nb + i / kFp8Block] = fs.base * rstd;
    } else if (a.code == kCodeI8 && in) {
      *reinterpret_cast<uint2*>(a.q + row + i) = quant_codes8(p.v, qs);
    }
  };
  if constexpr (HELD > 0) {
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      const int i = (h * LANES + l) * 8;
      finish(held[h], i, i < d);
    }
  } else {
    for (uint32_t i0 = 0; i0 < static_cast<uint32_t>(d); i0 += LANES * 8) {
      const uint32_t i = i0 + l * 8;
      const bool in = i < static_cast<uint32_t>(d);
      Piece p{};
      if (in) {
        if constexpr (R != kNone) p = load8<R == kBf16>(a.residual_out, row + i);
        else p = load8<X == kBf16>(a.x, row + i);
        weigh(p, unpack8(a.weight_bf16, load8_raw(a.weight_bf16, a.weight, i)));
      }
      finish(p, static_cast<int>(i), in);
    }
  }
  if (a.code == kCodeI8 && l == 0) a.s[t] = qs.scale * rstd;
}

template <Kind X, Kind R>
void launch_norm_rows(const NormArgs& a, hipStream_t stream) {
  const dim3 block(kThreads);
  const int pieces = a.d / 8;
  auto grid = [&](int lanes) { return dim3((static_cast<unsigned>(a.T) * lanes + kThreads - 1) / kThreads); };
  if (pieces <= 64) hipLaunchKernelGGL((rmsnorm<X, R, 64, 1>), grid(64), block, 0, stream, a);
  else if (pieces <= 128) hipLaunchKernelGGL((rmsnorm<X, R, 128, 1>), grid(128), block, 0, stream, a);
  else if (pieces <= 256) hipLaunchKernelGGL((rmsnorm<X, R, 256, 1>), grid(256), block, 0, stream, a);
  else if (pieces <= 512) hipLaunchKernelGGL((rmsnorm<X, R, 256, 2>), grid(256), block, 0, stream, a);
  else if (pieces <= 1024) hipLaunchKernelGGL((rmsnorm<X, R, 256, 4>), grid(256), block, 0, stream, a);
  else if (pieces <= 2048) hipLaunchKernelGGL((rmsnorm<X, R, 256, kMaxHeld>), grid(256), block, 0, stream, a);
  else hipLaunchKernelGGL((rmsnorm<X, R, 256, 0>), grid(256), block, 0, stream, a);
}

// ---- quantiser ------------------------------------------------------------------------
// 16 lanes take the 128 columns of a block, eight values each; n blocks from block `first`, nb in a row.
// 8191 x 2880 fp32: 17 us, 7 TB/s, so part of the rows comes from the last-level cache.
constexpr int kBlocksPer = kThreads / 16;

template <bool BF16>
__global__ __launch_bounds__(kThreads) void quantize_blocks(const void* __restrict__ x, int d, int nb, uint32_t first,
                                                            uint32_t n, uint8_t* __restrict__ q, float* __restrict__ s) {
  const uint32_t k = blockIdx.x * kBlocksPer + threadIdx.x / 16;
  const uint32_t b = first + min(k, n - 1);
  const uint32_t t = b / nb, i = (b - t * nb) * kFp8Block + threadIdx.x % 16 * 8;
  const bool in = k < n && i < static_cast<uint32_t>(d);
  const size_t at = static_cast<size_t>(t) * d + i;
  Piece p{};
  if (in) p = load8<BF16>(x, at);
  const Fp8Scale fs = fp8_scale(row16_max(piece_max(p)));
  if (!in) return;
  *reinterpret_cast<uint2*>(q + at) = fp8_codes8(p.v, fs);
  if (threadIdx.x % 16 == 0) s[b] = fs.base;
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& args, hipStream_t stream) {
  // a grid has fewer than 2^32 threads: at most 2^23 rows of a block each in a launch
  constexpr int kMost = 1 << 23;
  const int nb = (args.d + kFp8Block - 1) / kFp8Block;
  for (int t = 0; t < args.T; t += kMost) {
    NormArgs a = args;
    a.T = args.T - t < kMost ? args.T - t : kMost;
    const size_t at = static_cast<size_t>(t) * args.d;
    auto from = [&](const void* p, int bf16) { return p ? static_cast<const char*>(p) + at * (bf16 ? 2 : 4) : nullptr; };
    a.x = from(args.x, a.x_bf16);
    a.residual = from(args.residual, a.residual_bf16);
    a.residual_out = const_cast<char*>(from(args.residual_out, a.residual_bf16));
    a.y = const_cast<char*>(from(args.y, a.y_bf16));
    if (a.code != kCodeNone) {
      a.q = args.q + at;
      a.s = args.s + static_cast<size_t>(t) * (a.code == kCodeFp8 ? nb : 1);
    }
    const Kind r = !a.residual ? kNone : a.residual_bf16 ? kBf16 : kF32;
    if (a.x_bf16) {
      if (r == kNone) launch_norm_rows<kBf16, kNone>(a, stream);
      else if (r == kBf16) launch_norm_rows<kBf16, kBf16>(a, stream);
      else launch_norm_rows<kBf16, kF32>(a, stream);
    } else {
      if (r == kNone) launch_norm_rows<kF32, kNone>(a, stream);
      else if (r == kBf16) launch_norm_rows<kF32, kBf16>(a, stream);
      else launch_norm_rows<kF32, kF32>(a, stream);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.T < kMost) break;                     // t + kMost may pass int32
  }
  return hipSuccess;
}

hipError_t launch_quantize_blocks(const void* x, int bf16, int T, int d, uint8_t* q, float* s, hipStream_t stream) {
  constexpr uint32_t kMost = 1u << 27;          // blocks of 128 columns in a launch: 2^23 blocks of threads
  const int nb = (d + kFp8Block - 1) / kFp8Block;
  const uint32_t all = static_cast<uint32_t>(T) * nb;          // in int32 (moe_quantize_blocks_fp8)
  for (uint32_t b = 0; b < all; b += kMost) {
    const uint32_t n = all - b < kMost ? all - b : kMost;
    const dim3 grid((n + kBlocksPer - 1) / kBlocksPer), block(kThreads);
    if (bf16) hipLaunchKernelGGL((quantize_blocks<true>), grid, block, 0, stream, x, d, nb, b, n, q, s);
    else hipLaunchKernelGGL((quantize_blocks<false>), grid, block, 0, stream, x, d, nb, b, n, q, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
