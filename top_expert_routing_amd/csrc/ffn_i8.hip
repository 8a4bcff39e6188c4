// Grouped int8 products (moe_grouped_linear_i8, moe_grouped_ffn_i8) on the
// integer matrix instructions of gfx950.
//
// Rows are int8 codes with one scale per row, expert matrices packed int8 codes
// with one scale per output channel; the sums are exact int32 and the scales
// multiply them in fp32.  Three kinds of products share three kernels (few_i8, stream_i8, tile_i8):
//   kLinear  y = sx * sw * (xq . W)                                     -> bf16 or fp32
//   kGateUp  a = silu(sx sg (xq . Wg)) * (sx su (xq . Wu)), quantised per row and
//            128 columns (the columns of one tile)                      -> codes + scales
//   kDown    h = sw * sum over blocks of 128: sa[block] * (aq . Wd over the block)  -> bf16
// Quantising the SwiGLU product where it is made needs the largest magnitude of a
// row over the columns that share a scale, so a tile owns whole blocks: 128 columns.
// A scale for each 128 columns instead of one for the row keeps the product out of
// memory in 32 bits (N * I * 4 bytes written and read) and needs no launch in
// between; the price is one conversion and one fma per 128 products in kDown.
//
// v_mfma_i32_16x16x64_i8: lane 16 q + r holds the 16 codes K = 16 q .. 16 q + 15 of row
// r of either operand, which is what one KiB of a packed matrix holds in order.  The
// weight rows are the first operand, so in a 16x16 result lane 16 q + r has token
// row r and the output columns 4 q .. 4 q + 3.
#include <type_traits>

#include "common.h"
#include "i8_plan.h"
#include "launch.h"
#include "quantize.h"
#include "tile_util.h"

namespace moe {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

using namespace i8;

static_assert(kLanes == kWave, "one wavefront");
constexpr int kMaxGroups = 2 * 512 + 256;

struct ProductArgs {
  const void* x;           // few_i8<kGateUp>: bf16 tokens [n_x][K], in place of a and as
  const float* af;         // few_i8<kDown>: the SwiGLU product [n_rows][K], in place of a and as
  const int8_t* a;         // codes of the rows: [n_x][K]; kDown: [n_rows][K]
  const float* as;         // their scales: [n_x]; kDown: [ceil(K / 128)][n_rows]
  const int8_t *w0, *w1;   // packed matrices [E+S][cols][K] (w1: up rows of kGateUp)
  const float *s0, *s1;    // channel scales [E+S][cols]
  const int* x_rows;       // row list (nullptr: sorted row n reads row n)
  const int* offs;
  void* out;               // [n_rows][cols]: values, kGateUp: codes
  float* out_scale;        // kGateUp: [ceil(cols / 128)][n_rows]
  int n_x, n_rows, K, cols;
  int G, E, nseg;
};

__device__ __forceinline__ int src_row(const ProductArgs& p, int n) {
  return p.x_rows ? min(max(p.x_rows[n], 0), p.n_x - 1) : n;
}

__device__ __forceinline__ i32x4 mfma_i8(const uint4& w, const uint4& x, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), c, 0, 0, 0);
}

// Scale of a block of the SwiGLU product and the factor of its codes.  The products carry
// relative errors of b = (9.2 + 2.2 max(0, -g)) * 2^-23 anyhow (silu_mul), and so does the
// scale, their largest one / 127; so codes are rounded from v * (1 / scale) without the exact
// quotient's correction, which adds 3.5 * 2^-23.  A code moves only where its quotient lies within
// 127 times the sum of the three of a border (2^-16 * (22 + 2.2 * (n + m)) codes, libmoe_int8.h).
struct BlockScale {
  float scale, r;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) * (1.0f / 127.0f);
  if (amax_bits >= 0x7f800000u) return BlockScale{__builtin_nanf(""), 0.f};
  if (s < 0x1p-126f) return BlockScale{1.f, 0.f};
  return BlockScale{s, __builtin_amdgcn_rcpf(s)};
}
// Four codes: adding 1.5 * 2^23 rounds v * r to the nearest integer (halves to even) and
// leaves its two's complement in the low bits; |v * r| <= 127.0001.
__device__ __forceinline__ uint32_t block_codes(const float (&v)[4], float r) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(__builtin_fmaf(v[i], r, 12582912.0f));
  return low_bytes(c[0], c[1], c[2], c[3]);
}

// ---- small groups: weights stream from HBM into the matrix operands ----------------
// One block of eight waves per item (at most 16 * MF rows of a group, 128 output
// columns): each wave owns 16 columns (kGateUp: 16 gate rows and 16 up rows) and
// reads their weights once; the rows' codes are staged through LDS, 512 of K at a
// time, double buffered, and shared by the waves.
// Bound by the weights' bytes: 128 tokens x 8 of 64 experts, 2048 -> 1024, 137 MB in 28 us
// (4.8 TB/s); an FFN of 1088 tokens x 4 of 128 experts, 2880 x 2880, whose used experts'
// weights are 2.7 GB, 551 us (4.95 TB/s, the rate of a copy).  Asking for a step's next
// weights as soon as it is multiplied, instead of a chunk's together, changes 1 % either
// way; loads without the branches of a chunk past K are 2 % slower.
constexpr int kThreadsS = 512;
constexpr int kWavesS = kThreadsS / kWave;
constexpr int kChunk = 512;
constexpr int kPitch = kChunk + 16;  // bytes of a staged row: 16 rows start in 16 different bank groups

template <int MF, Mode M, class Out>
__global__ __launch_bounds__(kThreadsS, 4) void stream_i8(ProductArgs p) {
  constexpr int BM = 16 * MF;
  constexpr int NF = M == kGateUp ? 2 : 1;
  constexpr int U = kChunk / kStep;
  constexpr int VPR = kChunk / 16;                          // 16-byte pieces of a staged row
  constexpr int APT = BM * VPR / kThreadsS;                 // pieces per thread
  constexpr int BPC = kChunk / kBlock;                      // blocks of 128 in a chunk
  static_assert(BM * VPR % kThreadsS == 0, "whole pieces per thread");
  __shared__ __attribute__((aligned(16))) int8_t As[2][BM * kPitch];
  __shared__ float Ss[M == kDown ? 2 : 1][M == kDown ? BPC * BM : 1];
  __shared__ uint32_t amax[M == kGateUp ? kWavesS : 1][M == kGateUp ? BM : 1];

  const Item it = find_item(p, BM, (p.cols + kBlock - 1) / kBlock);
  if (it.rows == 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  const int l16 = lane & 15, q = lane >> 4;
  const int K = p.K, cols = p.cols;
  const int col0 = it.chunk * kBlock + wave * 16;
  const bool live = col0 < cols;                            // cols % 64 == 0: all 16 columns or none
  const size_t rb = static_cast<size_t>(it.expert) * cols + (live ? col0 : cols - 16);
  const int8_t* bp[NF];
  bp[0] = p.w0 + rb * K + lane * 16;
  if constexpr (NF == 2) bp[1] = p.w1 + rb * K + lane * 16;

  const int8_t* arow[APT];
  uint4 stage[APT];
  float sstage = 0.f;
#pragma unroll
  for (int s = 0; s < APT; ++s) {
    const int r = (threadIdx.x + s * kThreadsS) / VPR;
    arow[s] = r < it.rows ? p.a + static_cast<size_t>(M == kDown ? it.row(r) : src_row(p, it.row(r))) * K : nullptr;
  }
  auto load_a = [&](int c) {
#pragma unroll
    for (int s = 0; s < APT; ++s) {
      const int k = c * kChunk + (threadIdx.x + s * kThreadsS) % VPR * 16;
      stage[s] = arow[s] && k < K ? *reinterpret_cast<const uint4*>(arow[s] + k) : make_uint4(0, 0, 0, 0);
    }
    if constexpr (M == kDown) {
      const int r = threadIdx.x % BM, b = c * BPC + threadIdx.x / BM;
      sstage = threadIdx.x < BPC * BM && r < it.rows && b * kBlock < K
                   ? p.as[static_cast<size_t>(b) * p.n_rows + it.row(r)] : 0.f;
    }
  };
  auto store_a = [&](int buf) {
#pragma unroll
    for (int s = 0; s < APT; ++s) {
      const int i = threadIdx.x + s * kThreadsS;
      *reinterpret_cast<uint4*>(&As[buf][(i / VPR) * kPitch + (i % VPR) * 16]) = stage[s];
    }
    if constexpr (M == kDown)
      if (threadIdx.x < BPC * BM) Ss[buf][threadIdx.x] = sstage;
  };

  i32x4 acc[MF][NF];
  f32x4 facc[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    facc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  }
  const int nc = (K + kChunk - 1) / kChunk;
  load_a(0);
  store_a(0);
  for (int c = 0; c < nc; ++c) {
    uint4 b[U][NF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kk = c * kChunk + u * kStep;                // K % 64 == 0: whole steps
#pragma unroll
      for (int j = 0; j < NF; ++j)
        b[u][j] = kk < K ? *reinterpret_cast<const uint4*>(bp[j] + static_cast<size_t>(kk) * 16) : make_uint4(0, 0, 0, 0);
    }
    const bool more = c + 1 < nc;
    if (more) load_a(c + 1);
    __syncthreads();                                        // chunk c of the rows is staged
    const int8_t* as = As[c & 1] + l16 * kPitch + 16 * q;
    if constexpr (M == kDown) {
#pragma unroll
      for (int u = 0; u < U; u += 2)
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          const uint4 a0 = *reinterpret_cast<const uint4*>(as + 16 * i * kPitch + u * kStep);
          const uint4 a1 = *reinterpret_cast<const uint4*>(as + 16 * i * kPitch + (u + 1) * kStep);
          const i32x4 t = mfma_i8(b[u + 1][0], a1, mfma_i8(b[u][0], a0, i32x4{0, 0, 0, 0}));
          const float s = Ss[c & 1][(u / 2) * BM + 16 * i + l16];
#pragma unroll
          for (int r = 0; r < 4; ++r) facc[i][r] = __builtin_fmaf(static_cast<float>(t[r]), s, facc[i][r]);
        }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          const uint4 av = *reinterpret_cast<const uint4*>(as + 16 * i * kPitch + u * kStep);
#pragma unroll
          for (int j = 0; j < NF; ++j) acc[i][j] = mfma_i8(b[u][j], av, acc[i][j]);
        }
    }
    if (more) store_a((c + 1) & 1);                         // last read before this chunk's barrier
  }

  const int n = col0 + 4 * q;
  const size_t so = static_cast<size_t>(it.expert) * cols + (live ? n : 0);
  const f32x4 w0 = *reinterpret_cast<const f32x4*>(p.s0 + so);
  if constexpr (M == kGateUp) {
    const f32x4 w1 = *reinterpret_cast<const f32x4*>(p.s1 + so);
    float v[MF][4];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = 16 * i + l16;
      const float sx = m < it.rows ? p.as[src_row(p, it.row(m))] : 0.f;
      uint32_t big = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[i][r] = silu_mul(static_cast<float>(acc[i][0][r]) * (sx * w0[r]), static_cast<float>(acc[i][1][r]) * (sx * w1[r]));
        big = max(big, abs_bits(v[i][r]));
      }
      big = max(big, static_cast<uint32_t>(__shfl_xor(static_cast<int>(big), 16, kWave)));
      big = max(big, static_cast<uint32_t>(__shfl_xor(static_cast<int>(big), 32, kWave)));
      if (q == 0) amax[wave][m] = live ? big : 0u;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = 16 * i + l16;
      if (m >= it.rows) continue;
      uint32_t big = amax[0][m];
#pragma unroll
      for (int w = 1; w < kWavesS; ++w) big = max(big, amax[w][m]);
      const BlockScale qs = block_scale(big);
      const int row = it.row(m);
      if (live)
        *reinterpret_cast<uint32_t*>(static_cast<int8_t*>(p.out) + static_cast<size_t>(row) * cols + n) =
            block_codes(v[i], qs.r);
      if (wave == 0 && q == 0) p.out_scale[static_cast<size_t>(it.chunk) * p.n_rows + row] = qs.scale;
    }
  } else {
    if (!live) return;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = 16 * i + l16;
      if (m >= it.rows) continue;
      const int row = it.row(m);
      float v[4];
      if constexpr (M == kDown) {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = facc[i][r] * w0[r];
      } else {
        const float sx = p.as[src_row(p, row)];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = static_cast<float>(acc[i][0][r]) * (sx * w0[r]);
      }
      store4(static_cast<Out*>(p.out) + static_cast<size_t>(row) * cols + n, v);
    }
  }
}

// ---- few rows: 16 columns per block, K split over its waves --------------------------
// With few rows (one token's experts, a small dense batch) 128-column items are too few
// to draw the weights through every CU, so an item is 16 columns (kGateUp: 16 gate and 16
// up rows) of at most 16 rows and the eight waves split K; their sums are joined through
// LDS.  A wave's first weights are requested before anything else happens.
// Bound by that chain (group offsets, weights, rows, join) around one burst of weights: one
// token's FFN, 8 experts of 2048 x 1024 (50 MB), 16.6 us; 5 rows x 2048 -> 2048 (4 MB) 3.9.
// The FFN's quantisations move to where codes are used, because a block no longer holds
// the columns that share a scale, and each block repeats them (16 rows at most):
//   * kGateUp reads the bf16 tokens: a wave's slice of K gives part of a row's largest
//     magnitude, LDS the rest; then the slice's codes are made next to the weights' loads.
//     This saves the launch that quantises the tokens.
//   * it writes the SwiGLU product in fp32 (N * I * 4 bytes, at most 80 KiB here), and
//     kDown's waves, each on whole blocks of 128 columns, quantise it as they read it.
constexpr int kFewSteps = 4;            // K steps in flight per wave
constexpr int kSplit = kWavesS;

// Codes of the eight values of row piece v, as quant_codes8, per-lane scales.
__device__ __forceinline__ uint4 bf16_codes(const uint4& lo, const uint4& hi, const QuantScale& qs) {
  auto eight = [&](const uint4& u) MOE_INLINE {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return quant_codes8(v, qs);
  };
  const uint2 a = eight(lo), b = eight(hi);
  return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ uint32_t bf16_max(const uint4& u) {      // largest magnitude's fp32 bits
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
  return m;
}
template <int NC, Mode M, class Out>
__global__ __launch_bounds__(kThreadsS, NC == 1 ? 4 : 2) void few_i8(ProductArgs p) {
  constexpr int NF = M == kGateUp ? 2 * NC : NC, U = kFewSteps;   // j < NC: gate or only, j >= NC: up
  __shared__ i32x4 part[kSplit][NF][kWave];
  __shared__ uint32_t amax[kSplit][16];
  const Item it = find_item(p, 16, p.cols / (16 * NC));
  if (it.rows == 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  const int l16 = lane & 15, q = lane >> 4;
  const int K = p.K, cols = p.cols;
  // this wave's K: whole blocks of 128, dealt in equal runs
  const int run = ((K + kBlock - 1) / kBlock + kSplit - 1) / kSplit * kBlock;
  const int k0 = min(K, wave * run), k1 = min(K, k0 + run);
  const size_t rb = static_cast<size_t>(it.expert) * cols + it.chunk * 16 * NC;
  const int8_t* wp[NF];                                     // wave-uniform; a lane's 16 bytes are its `lane`-th
#pragma unroll
  for (int j = 0; j < NF; ++j) wp[j] = (j < NC ? p.w0 : p.w1) + (rb + 16 * (j % NC)) * K;
  uint4 w[U][NF];
  // Loads without branches, so that the waits count them one by one: a step past this wave's
  // run loads the matrix's last one (where K is short), which is not multiplied.
  auto step_at = [&](int k, int u) MOE_INLINE { return static_cast<size_t>(min(k + u * kStep, K - kStep)); };
  auto load_w = [&](int k, int u0, int u1) MOE_INLINE {
#pragma unroll
    for (int u = u0; u < u1; ++u)
#pragma unroll
      for (int j = 0; j < NF; ++j) w[u][j] = reinterpret_cast<const uint4*>(wp[j] + step_at(k, u) * 16)[lane];
  };
  // this lane's row (lanes past the rows repeat the last one) and its 16 values of each K step: bf16, fp32 or codes
  const int row = it.row(min(l16, it.rows - 1));
  constexpr int PIECES = M == kGateUp ? 2 : M == kDown ? 4 : 1;
  uint4 x[U][PIECES];
  const uint8_t* xr = nullptr;
  auto load_x = [&](int k) MOE_INLINE {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < PIECES; ++i) x[u][i] = reinterpret_cast<const uint4*>(xr + step_at(k, u) * PIECES)[i];
  };
  // A wave's loads return in order, so the first rows are asked for among the first weights: behind them
  // (17.8 us for one token's FFN) what the rows are still to go through would wait for every weight.
  int src = row;
  if constexpr (M == kDown) {
    xr = reinterpret_cast<const uint8_t*>(p.af + static_cast<size_t>(row) * K + 16 * q);
    load_x(k0);
    __builtin_amdgcn_sched_barrier(0);
    load_w(k0, 0, U);
  } else {
    const int listed = *(p.x_rows ? p.x_rows + row : p.offs);
    load_w(k0, 0, U / 2);
    __builtin_amdgcn_sched_barrier(0);
    if (p.x_rows) src = min(max(listed, 0), p.n_x - 1);
    const uint8_t* base = static_cast<const uint8_t*>(M == kGateUp ? p.x : p.a);
    xr = base + (static_cast<size_t>(src) * K + 16 * q) * (M == kGateUp ? 2 : 1);
    load_x(k0);
    __builtin_amdgcn_sched_barrier(0);
    load_w(k0, U / 2, U);
  }
  __builtin_amdgcn_sched_barrier(0);

  QuantScale qs{1.f, 1.f, 1.f, 1.f};                        // kGateUp: of this lane's token
  if constexpr (M == kGateUp) {
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) m = max(m, max(bf16_max(x[u][0]), bf16_max(x[u][1])));   // repeated steps change nothing
    for (int k = k0 + U * kStep; k < k1; k += kStep) {
      const uint4* v = reinterpret_cast<const uint4*>(xr + static_cast<size_t>(k) * 2);
      m = max(m, max(bf16_max(v[0]), bf16_max(v[1])));
    }
    m = max_over_q(m);
    if (q == 0) amax[wave][l16] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSplit; ++i) m = max(m, amax[i][l16]);
    qs = quant_scale(m);
  }
  i32x4 acc[NF];
  f32x4 facc[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) facc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < NF; ++j) acc[j] = i32x4{0, 0, 0, 0};
  for (int k = k0; k < k1; k += U * kStep) {
    if (k != k0) {
      load_x(k);
      load_w(k, 0, U);
    }
    if constexpr (M == kDown) {
      // blocks of 128 columns of the fp32 product: their scale, then their codes (columns past K are zeros)
#pragma unroll
      for (int u = 0; u < U; u += 2) {
        if (k + u * kStep >= k1) break;
        float v[8][4];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f32x4 f = __builtin_bit_cast(f32x4, x[u + i / 4][i % 4]);
          if (i >= 4 && k + (u + 1) * kStep >= k1) f = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            v[i][r] = f[r];
            m = max(m, abs_bits(f[r]));
          }
        }
        const BlockScale bs = block_scale(max_over_q(m));
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = block_codes(v[i], bs.r);
        const uint4 a0 = make_uint4(c[0], c[1], c[2], c[3]), a1 = make_uint4(c[4], c[5], c[6], c[7]);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          const i32x4 t = mfma_i8(w[u + 1][j], a1, mfma_i8(w[u][j], a0, i32x4{0, 0, 0, 0}));
#pragma unroll
          for (int r = 0; r < 4; ++r) facc[j][r] = __builtin_fmaf(static_cast<float>(t[r]), bs.scale, facc[j][r]);
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k + u * kStep >= k1) break;
        uint4 a = x[u][0];
        if constexpr (M == kGateUp) a = bf16_codes(x[u][0], x[u][1], qs);
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[j] = mfma_i8(w[u][j], a, acc[j]);
      }
    }
  }
  // join: float sums in wave order, so that a result does not depend on timing; wave j
  // takes column block j
#pragma unroll
  for (int j = 0; j < NF; ++j) part[wave][j][lane] = M == kDown ? __builtin_bit_cast(i32x4, facc[j % NC]) : acc[j];
  __syncthreads();
  if (wave >= NC || l16 >= it.rows) return;
  auto joined = [&](int j) MOE_INLINE {
    f32x4 v;
    if constexpr (M == kDown) {
      v = __builtin_bit_cast(f32x4, part[0][j][lane]);
#pragma unroll
      for (int i = 1; i < kSplit; ++i) v += __builtin_bit_cast(f32x4, part[i][j][lane]);
    } else {
      i32x4 t = part[0][j][lane];
#pragma unroll
      for (int i = 1; i < kSplit; ++i) t += part[i][j][lane];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = static_cast<float>(t[r]);
    }
    return v;
  };
  const int n = (it.chunk * NC + wave) * 16 + 4 * q;
  const size_t so = static_cast<size_t>(it.expert) * cols + n;
  const f32x4 s0 = *reinterpret_cast<const f32x4*>(p.s0 + so), g = joined(wave);
  float v[4];
  if constexpr (M == kGateUp) {
    const f32x4 s1 = *reinterpret_cast<const f32x4*>(p.s1 + so), u = joined(NC + wave);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = silu_mul(g[r] * (qs.scale * s0[r]), u[r] * (qs.scale * s1[r]));
  } else {
    const float sx = M == kLinear ? p.as[src] : 1.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = g[r] * (sx * s0[r]);
  }
  store4(static_cast<Out*>(p.out) + static_cast<size_t>(row) * cols + n, v);
}

// ---- large groups: LDS-tiled products ----------------------------------------------
// A persistent block (one per CU) walks its list of tiles: BM rows x 256 weight rows
// (kGateUp: 128 gate and the same 128 up rows).  K advances 64 codes a step through a
// ring of LDS stages that LDS-DMA loads fill ahead; the steps of all tiles form one
// stream, so the next tile's first steps load while this one finishes.
//   * rows: 64 bytes of a row per step, four 16-byte pieces; piece c of row r lies at slot
//     c ^ swz(r), so that the 16 rows of an operand read hit different banks.  A DMA
//     instruction fills 16 rows (lane -> row lane / 4, slot lane % 4).
//   * weights: a packed block (16 rows x 64 codes, 1 KiB) is copied as it is.
//   * what the epilogue and the next tile need from memory (the row list, the rows' and
//     the channels' scales) comes by DMA too, a tile ahead, because a load that the
//     compiler sees would make it wait for everything in flight.
// Waves: WM x WN, each MI x NJ blocks of 16x16 (TileCfg, TileLds: i8_plan.h); the 16-row blocks of the waves interleave,
// so the rows of a partial tile spread over them.
// 8191 x 2048 -> 4096 (fp32 out) takes 79 us, 1.74 POP/s; K = 8192 reaches 2.5.  The matrix
// cores are busy 43 % of the cycles, waves wait 41 %: the barrier of each 64-wide step, the
// first loads and the epilogue of a tile (some 7 us of 35) bound it.  An FFN of 4096 tokens x 8
// of 128 experts, 2048 x 768, 266 us: a fifth of it are the experts' weights coming from HBM
// (every tile on one expert's: 0.83 of the time), the rest ragged tiles and, in kDown, the
// conversion and fma for each product.  TileHalf (three stages) and kDown (two) wait for every load
// in flight before a step, so that cold weights show as the rest of an HBM access.  Not kept: waves of 128 x 128, sixteen waves, panels of
// 2 or 8 column chunks, tiles of equal height within a group, skipping the operand reads of
// empty blocks, one barrier for two steps (it has to wait for every load and read: 81 us and
// 278); each within 2 % or slower.
__device__ __forceinline__ int swz(int r) { return ((r >> 1) ^ (r >> 2)) & 3; }

template <class C, Mode M, class Out>
__global__ __launch_bounds__(C::NT, C::BPC * C::NW / 4) void tile_i8(ProductArgs p) {
  using L = TileLds<C, M>;
  constexpr int MI = C::MI, NJ = C::NJ, WM = C::WM, WN = C::WN, NW = C::NW, NT = C::NT, BM = C::BM;
  constexpr int OUTC = M == kGateUp ? C::BN / 2 : C::BN;
  constexpr int GPT = (kMaxGroups + NT - 1) / NT;
  constexpr int kPanel = 4;                                    // column chunks that follow each other per m-tile
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int* wsum = reinterpret_cast<int*>(lds + L::PLAN);
  int* before = wsum + NW;                                     // m-tiles before group g
  int* offs = before + p.G + 1;
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4, wm = wave / WN, wn = wave % WN;
  const int K = p.K, cols = p.cols;

  for (int g = tid; g <= p.G; g += NT) offs[g] = p.offs[g];
  __syncthreads();
  {
    int cnt[GPT], sum = 0;
#pragma unroll
    for (int i = 0; i < GPT; ++i) {
      const int g = tid * GPT + i;
      cnt[i] = g < p.G ? group_rows(offs, p.n_rows, p.E, p.nseg, BM, g).nt : 0;
      sum += cnt[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int y = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += y;
    }
    if (lane == kWave - 1) wsum[wave] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int i = 0; i < wave; ++i) run += wsum[i];
#pragma unroll
    for (int i = 0; i < GPT; ++i) {
      const int g = tid * GPT + i;
      if (g < p.G) before[g] = run;
      run += cnt[i];
    }
    if (tid == NT - 1) before[p.G] = run;
    __syncthreads();
  }
  // XCD x (blocks are dealt round-robin) owns the x-th eighth of the list of tiles, so
  // that tiles which share weights or rows run in one L2; its blocks take them in turn
  const int nch = (cols + OUTC - 1) / OUTC;
  const int items = __builtin_amdgcn_readfirstlane(before[p.G]) * nch;
  const int per_xcd = static_cast<int>(gridDim.x) / kXcds;
  const int share = (items + kXcds - 1) / kXcds;
  const int first = static_cast<int>(blockIdx.x % kXcds) * share + static_cast<int>(blockIdx.x / kXcds);
  const int end = min(items, static_cast<int>(blockIdx.x % kXcds + 1) * share);
  const int n_my = first < end ? (end - first - 1) / per_xcd + 1 : 0;
  if (n_my == 0) return;
  auto item_of = [&](int i) MOE_INLINE -> Item {
    const int want = first + i * per_xcd;
    const int u = want / nch;
    int lo = 0, hi = p.G;                                      // last g with before[g] <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= u) lo = mid; else hi = mid;
    }
    const int nt = before[lo + 1] - before[lo];
    const int local = want - before[lo] * nch;
    const int panel = local / (kPanel * nt), rest = local - panel * kPanel * nt;
    const int pc = min(kPanel, nch - panel * kPanel);
    return uniform(group_tile(group_rows(offs, p.n_rows, p.E, p.nseg, BM, lo), lo, rest / pc, panel * kPanel + rest % pc,
                              BM, p.E, p.nseg));
  };

  // ---- the loads, STAGES - 1 steps ahead of the products
  const uint32_t lds0 = lds_address(lds);
  const int nsteps = K / kStep, nk = (nsteps + L::SUB - 1) / L::SUB;   // K steps and stages of a tile
  uint32_t ao[C::ADMA], ao_next[C::ADMA];                      // this lane's bytes from p.a: tile being loaded, tile after it
  const int8_t *bp[C::BDMA], *bp_next[C::BDMA];                // wave-uniform
  const float *sp = nullptr, *sp_next = nullptr;               // kDown: this lane's row's block scales
  // 4-byte loads of one value per row: lane 16 i + r of a wave has row r of the 16 rows of its
  // load i, so wave w's values are the w-th 16 * ADMA of ROWS
  const bool vlane = lane < 16 * C::ADMA;
  const int vrow = 16 * (wave + NW * (lane >> 4)) + l16;
  auto load_list = [&](const Item& it, int parity) MOE_INLINE {
    if (p.x_rows && vlane)
      dma4(p.x_rows + it.row(min(vrow, it.rows - 1)), lds0 + L::LIST + parity * L::ROWS + wave * L::WROWS);
  };
  // Sources of a tile whose row list has arrived; requests its scales.
  auto aim = [&](const Item& it, int parity) MOE_INLINE {
    const int* list = reinterpret_cast<const int*>(lds + L::LIST + parity * L::ROWS + wave * L::WROWS);
    auto src = [&](int r, int slot) MOE_INLINE {
      return p.x_rows ? min(max(list[slot], 0), p.n_x - 1) : it.row(min(r, it.rows - 1));
    };
#pragma unroll
    for (int i = 0; i < C::ADMA; ++i) {
      const int r = 16 * (wave + NW * i) + (lane >> 2);
      ao_next[i] = static_cast<uint32_t>(src(r, 16 * i + (lane >> 2))) * K + 16 * ((lane & 3) ^ swz(r));
    }
    const int n0 = it.chunk * OUTC;
    const size_t e0 = static_cast<size_t>(it.expert) * cols;
#pragma unroll
    for (int i = 0; i < C::BDMA; ++i) {
      const int b = wave + NW * i;                             // 16-row block of the tile
      const bool up = M == kGateUp && b >= C::BN / 32;
      const int n = min(n0 + 16 * (up ? b - C::BN / 32 : b), cols - 16);   // past the columns: read, never stored
      bp_next[i] = (up ? p.w1 : p.w0) + (e0 + n) * K;
    }
    if (wave == 0) {
      const bool up = M == kGateUp && lane >= 32;
      const int n = min(n0 + 4 * (M == kGateUp ? lane & 31 : lane), cols - 4);
      dma16((up ? p.s1 : p.s0) + e0 + n, lds0 + L::SB + parity * 1024);
    }
    if constexpr (M == kDown) sp_next = p.as + it.row(min(vrow, it.rows - 1));
    else if (vlane) dma4(p.as + src(vrow, lane), lds0 + L::SA + parity * L::ROWS + wave * L::WROWS);
  };
  int ikt = 0, islot = 0;                                      // the stage requested next: of its tile, ring slot
  auto turn = [&]() MOE_INLINE {                               // go on with the next tile
    ikt = 0;
#pragma unroll
    for (int i = 0; i < C::ADMA; ++i) ao[i] = ao_next[i];
#pragma unroll
    for (int i = 0; i < C::BDMA; ++i) bp[i] = bp_next[i];
    sp = sp_next;
  };
  constexpr int PER = L::SUB * (C::ADMA + C::BDMA);            // loads of a stage per wave (kDown: and one of scales)
  auto load = [&](int i) MOE_INLINE {                          // the i-th of them
    const int s = i / (C::ADMA + C::BDMA), n = i % (C::ADMA + C::BDMA);
    const int kt = min(ikt * L::SUB + s, nsteps - 1);          // steps past K: loaded again, not used
    const uint32_t st = lds0 + islot * L::STAGE + wave * 1024;
    if (n < C::ADMA) dma16(p.a + kt * kStep, ao[n], st + s * L::A + n * NW * 1024);
    else dma16(bp[n - C::ADMA] + static_cast<size_t>(kt) * 1024, lane * 16, st + L::SUB * L::A + s * L::B + (n - C::ADMA) * NW * 1024);
  };
  // kLinear, kGateUp take K steps in pairs (two register sets), an odd last one with an empty step
  const int stages = M == kDown ? nk : (nk + 1) & ~1;
  auto loaded = [&]() MOE_INLINE {
    islot = islot + 1 == L::STAGES ? 0 : islot + 1;
    if (++ikt == stages) turn();
  };
  auto load_scales = [&]() MOE_INLINE {
    if constexpr (M == kDown)
      if (vlane)
        dma4(sp + static_cast<size_t>(ikt) * p.n_rows, lds0 + islot * L::STAGE + L::SUB * (L::A + L::B) + wave * L::WROWS);
  };
  Item cur = item_of(0), nxt = n_my > 1 ? item_of(1) : cur;
  load_list(cur, 0);
  load_list(nxt, 1);
  wait_loads_barrier<0>();
  aim(cur, 0);
  turn();
#pragma unroll 1
  for (int s = 0; s < L::AHEAD; ++s) {                         // stages > AHEAD (TileLds, kTileMinK)
    load_scales();
#pragma unroll
    for (int i = 0; i < PER; ++i) load(i);
    loaded();
  }

  // ---- compute side
  const int aoff = 16 * wm * kStep + l16 * kStep + 16 * (q ^ swz(l16));   // 16-row blocks do not change swz
  int cslot = 0;
  auto next_stage = [&]() MOE_INLINE {
    const uint8_t* st = lds + cslot * L::STAGE;
    cslot = cslot + 1 == L::STAGES ? 0 : cslot + 1;
    return st;
  };
  auto bfrag = [&](const uint8_t* st, int s, int j) MOE_INLINE {
    const int b = M == kGateUp ? (j < NJ / 2 ? wn * (NJ / 2) + j : C::BN / 32 + wn * (NJ / 2) + j - NJ / 2) : wn * NJ + j;
    return *reinterpret_cast<const uint4*>(st + L::SUB * L::A + s * L::B + b * 1024 + lane * 16);
  };
  auto afrag = [&](const uint8_t* st, int s, int i) MOE_INLINE {
    return *reinterpret_cast<const uint4*>(st + s * L::A + aoff + 16 * WM * i * kStep);
  };
  // kLinear, kGateUp: a step's operands are read from LDS while the step before multiplies
  uint4 fa[M == kDown ? 1 : MI], fb[2][M == kDown ? 1 : NJ];
  if constexpr (M != kDown) {
    wait_loads_barrier<(L::AHEAD - 1) * PER>();
    const uint8_t* st = next_stage();
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[i] = afrag(st, 0, i);
#pragma unroll
    for (int j = 0; j < NJ; ++j) fb[0][j] = bfrag(st, 0, j);
  }
#pragma unroll 1
  for (int cr = 0; cr < n_my; ++cr) {
    const Item it = cur;
    const int par = cr & 1;
    // every wave is done with tile cr - 1: its lists and scales make room for tile cr + 1
    lds_barrier();
    aim(nxt, par ^ 1);
    cur = nxt;
    if (cr + 2 < n_my) nxt = item_of(cr + 2);
    load_list(nxt, par);
    i32x4 acc[M == kDown ? 1 : MI][M == kDown ? 1 : NJ];
    f32x4 facc[M == kDown ? MI : 1][M == kDown ? NJ : 1];
    if constexpr (M == kDown) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) facc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    } else {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    }
    const int blocks = (it.rows + 15) >> 4;                    // 16-row blocks with rows
    const int nv = __builtin_amdgcn_readfirstlane(min(MI, max(0, (blocks - wm + WM - 1) / WM)));   // of them this wave's
    if constexpr (M == kDown) {
      // the K loop over the first NI of the wave's 16-row blocks (one copy for each: a partial tile
      // skips its empty blocks' products and their scaling; 269 to 266 us for 128 ragged groups of 256)
      auto run = [&](auto ni) MOE_INLINE {
        constexpr int NI = decltype(ni)::value;
#pragma unroll 1
        for (int kt = 0; kt < nk; ++kt) {
          wait_loads_barrier<(L::AHEAD - 1) * PER>();          // this stage is complete, every wave is past the last one
          load_scales();
#pragma unroll
          for (int i = 0; i < PER; ++i) load(i);
          loaded();
          const uint8_t* st = next_stage();
          if constexpr (NI > 0) {
            const bool two = 2 * kt + 1 < nsteps;
            const float* sc = reinterpret_cast<const float*>(st + L::SUB * (L::A + L::B));
            uint4 a0[NI], a1[NI];
            float s[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              a0[i] = afrag(st, 0, i);
              a1[i] = two ? afrag(st, 1, i) : make_uint4(0, 0, 0, 0);
              const int blk = wm + WM * i;
              s[i] = sc[(blk % NW) * (16 * C::ADMA) + (blk / NW) * 16 + l16];
            }
            // the sums of column block j are scaled into facc while block j + 1 multiplies,
            // and the operands of block j + 2 are read
            uint4 b0 = bfrag(st, 0, 0), b1 = bfrag(st, 1, 0), d0 = bfrag(st, 0, 1), d1 = bfrag(st, 1, 1);
            i32x4 t[2][NI];
#pragma unroll
            for (int j = 0; j <= NJ; ++j) {
              uint4 c0, c1;
              if (j + 2 < NJ) c0 = bfrag(st, 0, j + 2), c1 = bfrag(st, 1, j + 2);
              if (j < NJ) {
#pragma unroll
                for (int i = 0; i < NI; ++i) t[j & 1][i] = mfma_i8(b0, a0[i], i32x4{0, 0, 0, 0});
#pragma unroll
                for (int i = 0; i < NI; ++i) t[j & 1][i] = mfma_i8(b1, a1[i], t[j & 1][i]);
              }
              if (j > 0) {
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                  for (int r = 0; r < 4; ++r)
                    facc[i][j - 1][r] = __builtin_fmaf(static_cast<float>(t[(j - 1) & 1][i][r]), s[i], facc[i][j - 1][r]);
              }
              if (j > 0 && j < NJ) {
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // the reads first, then one product, four
#pragma unroll
                for (int i = 0; i < 2 * NI; ++i) {                   // conversions or sums, one product, ...
                  __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                  __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
                }
              }
              __builtin_amdgcn_sched_barrier(0);
              b0 = d0, b1 = d1, d0 = c0, d1 = c1;
            }
          }
        }
      };
      static_assert(MI == 4, "one copy for each number of blocks");
      if (nv == 4) run(std::integral_constant<int, 4>{});
      else if (nv == 3) run(std::integral_constant<int, 3>{});
      else if (nv == 2) run(std::integral_constant<int, 2>{});
      else if (nv == 1) run(std::integral_constant<int, 1>{});
      else run(std::integral_constant<int, 0>{});
    } else {
      // One step on the operands fa, b (n: 16-row blocks to multiply); reads the next step's into
      // fa (each block after its last use) and bn.
      auto step = [&](int n, uint4 (&b)[NJ], uint4 (&bn)[NJ]) MOE_INLINE {
        // the next stage is complete in LDS, and every wave is past the step before this one
        wait_loads_barrier<(L::AHEAD - 2) * PER>();
        const uint8_t* st = next_stage();
#pragma unroll
        for (int i = 0; i < MI; ++i) {
#pragma unroll
          for (int j = i * NJ / MI; j < (i + 1) * NJ / MI; ++j) bn[j] = bfrag(st, 0, j);
          if (i < n) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = mfma_i8(b[j], fa[i], acc[i][j]);
          }
#pragma unroll
          for (int l = i * PER / MI; l < (i + 1) * PER / MI; ++l) load(l);
          fa[i] = afrag(st, 0, i);
          __builtin_amdgcn_sched_barrier(0);
        }
        loaded();
      };
#pragma unroll 1
      for (int kt = 0; kt < nk; kt += 2) {
        step(nv, fb[0], fb[1]);
        step(kt + 1 < nk ? nv : 0, fb[1], fb[0]);
      }
    }

    // ---- epilogue
    const float* sa = reinterpret_cast<const float*>(lds + L::SA + par * L::ROWS);
    const float* sb = reinterpret_cast<const float*>(lds + L::SB + par * 1024);
    const int n0 = it.chunk * OUTC;
    if constexpr (M == kGateUp) {
      uint32_t* mx = reinterpret_cast<uint32_t*>(lds + L::MAX);
      float v[MI][NJ / 2][4];
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int blk = wm + WM * i;
        const float sx = sa[(blk % NW) * (16 * C::ADMA) + (blk / NW) * 16 + l16];
        uint32_t big = 0;
#pragma unroll
        for (int j = 0; j < NJ / 2; ++j) {
          const int c = 16 * (wn * (NJ / 2) + j) + 4 * q;
          const f32x4 w0 = *reinterpret_cast<const f32x4*>(sb + c), w1 = *reinterpret_cast<const f32x4*>(sb + 128 + c);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            v[i][j][r] = silu_mul(static_cast<float>(acc[i][j][r]) * (sx * w0[r]),
                                  static_cast<float>(acc[i][NJ / 2 + j][r]) * (sx * w1[r]));
            if (n0 + c < cols) big = max(big, abs_bits(v[i][j][r]));
          }
        }
        big = max(big, static_cast<uint32_t>(__shfl_xor(static_cast<int>(big), 16, kWave)));
        big = max(big, static_cast<uint32_t>(__shfl_xor(static_cast<int>(big), 32, kWave)));
        if (q == 0) mx[wn * BM + 16 * blk + l16] = big;
      }
      lds_barrier();
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int m = 16 * (wm + WM * i) + l16;
        if (16 * (wm + WM * i) >= it.rows) continue;           // wave-uniform; the exchange below needs every lane
        uint32_t big = mx[m];
#pragma unroll
        for (int w = 1; w < WN; ++w) big = max(big, mx[w * BM + m]);
        const BlockScale qs = block_scale(big);
        static_assert(NJ / 2 == 4, "one 16-byte store per row and lane");
        uint32_t d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = block_codes(v[i][j], qs.r);
        transpose_rows(d);                                     // now lane 16 q + r: the 16 columns of block q
        if (m >= it.rows) continue;
        const int row = it.row(m), n = n0 + 16 * (wn * 4 + q);
        if (wn == 0 && q == 0) p.out_scale[static_cast<size_t>(it.chunk) * p.n_rows + row] = qs.scale;
        if (n < cols)
          *reinterpret_cast<uint4*>(static_cast<int8_t*>(p.out) + static_cast<size_t>(row) * cols + n) =
              make_uint4(d[0], d[1], d[2], d[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int blk = wm + WM * i, m = 16 * blk + l16;
        if (16 * blk >= it.rows) continue;                     // wave-uniform
        float sx = 1.f;
        if constexpr (M == kLinear) sx = sa[(blk % NW) * (16 * C::ADMA) + (blk / NW) * 16 + l16];
        const bool in = m < it.rows;
        Out* orow = static_cast<Out*>(p.out) + static_cast<size_t>(it.row(in ? m : 0)) * cols + n0;
        auto values = [&](int j, float (&v)[4]) MOE_INLINE {
          const f32x4 w0 = *reinterpret_cast<const f32x4*>(sb + 16 * (wn * NJ + j) + 4 * q);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if constexpr (M == kDown) v[r] = facc[i][j][r] * w0[r];
            else v[r] = static_cast<float>(acc[i][j][r]) * (sx * w0[r]);
          }
        };
        if constexpr (sizeof(Out) == 4) {
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            float v[4];
            values(j, v);
            const int c = 16 * (wn * NJ + j) + 4 * q;
            if (in && n0 + c < cols) store4(orow + c, v);
          }
        } else {
          // bf16: two column blocks to 16 bytes a lane: row q = 2 a + b gets columns 8 b .. 8 b + 7 of block j + a
#pragma unroll
          for (int j = 0; j < NJ; j += 2) {
            float v[4], u[4];
            values(j, v);
            values(j + 1, u);
            uint32_t d[4] = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3])};
            swap32(d[0], d[2]);
            swap32(d[1], d[3]);
            swap16(d[0], d[2]);
            swap16(d[1], d[3]);
            const int c = 16 * (wn * NJ + j + (q >> 1)) + 8 * (q & 1);
            if (in && n0 + c < cols) *reinterpret_cast<uint4*>(orow + c) = make_uint4(d[0], d[1], d[2], d[3]);
          }
        }
      }
    }
  }
  // the stages requested past the last tile land in LDS: not after this block has left it
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <Mode M, class Out>
void launch_few(const ProductArgs& p, const Plan& plan, hipStream_t stream) {
  const Launch l = launch_of(plan);
  const dim3 grid(l.x, l.y), block(kThreadsS);
  if (plan.width == 1) hipLaunchKernelGGL((few_i8<1, M, Out>), grid, block, 0, stream, p);
  else if (plan.width == 2) hipLaunchKernelGGL((few_i8<2, M, Out>), grid, block, 0, stream, p);
  else if constexpr (M != kGateUp) hipLaunchKernelGGL((few_i8<4, M, Out>), grid, block, 0, stream, p);
}

template <class Tile, Mode M, class Out>
void launch_tile(const ProductArgs& p, hipStream_t stream) {
  const int cus = (device_cus() + kXcds - 1) / kXcds * kXcds;
  const size_t lds = TileLds<Tile, M>::bytes(p.G);
  hipLaunchKernelGGL((tile_i8<Tile, M, Out>), dim3(cus * Tile::BPC), dim3(Tile::NT), lds, stream, p);
}

template <Mode M, class Out>
void launch_many(const ProductArgs& p, const Plan& plan, hipStream_t stream) {
  if (plan.kernel == Kernel::kStream) {
    const Launch l = launch_of(plan);
    const dim3 grid(l.x, l.y), block(kThreadsS);
    if (plan.width == 1) hipLaunchKernelGGL((stream_i8<1, M, Out>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((stream_i8<2, M, Out>), grid, block, 0, stream, p);
  } else if (plan.kernel == Kernel::kTileWide) {
    launch_tile<TileWide, M, Out>(p, stream);
  } else if constexpr (M != kDown) {
    launch_tile<TileHalf, M, Out>(p, stream);
  }
}

Sizes sizes_of(const ProductArgs& p) { return Sizes{p.n_rows, p.E, p.G - p.nseg * p.E, p.nseg, p.K, p.cols}; }

ProductArgs product_args(const GroupedI8& g, int K, int cols) {
  ProductArgs p{};
  p.x_rows = g.x_rows;
  p.offs = g.group_offsets;
  p.n_x = g.n_x;
  p.n_rows = g.n_rows;
  p.K = K;
  p.cols = cols;
  p.G = g.nseg * g.E + g.n_shared;
  p.E = g.E;
  p.nseg = g.nseg;
  return p;
}

// Workspace of the FFN: token codes and scales, SwiGLU codes and block scales.
struct FfnI8Layout {
  size_t xs, aq, as, total;   // byte offsets (the token codes start at 0)
};
FfnI8Layout ffn_i8_layout(int n_rows, int n_tokens, int d, int I) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  FfnI8Layout L;
  L.xs = up(static_cast<size_t>(n_tokens) * d);
  L.aq = L.xs + up(static_cast<size_t>(n_tokens) * 4);
  L.as = L.aq + up(static_cast<size_t>(n_rows) * I * (few(n_rows, I) ? 4 : 1));   // few rows: in fp32
  L.total = L.as + up(static_cast<size_t>((I + kBlock - 1) / kBlock) * n_rows * 4);
  return L;
}

}  // namespace

hipError_t launch_grouped_linear_i8(const GroupedI8& g, const int8_t* xq, const float* xs, int K, int O,
                                    const int8_t* w, const float* ws, int bf16, void* y, hipStream_t stream) {
  ProductArgs p = product_args(g, K, O);
  p.a = xq;
  p.as = xs;
  p.w0 = w;
  p.s0 = ws;
  p.out = y;
  const Plan plan = plan_linear(sizes_of(p));
  if (plan.kernel == Kernel::kFew) {
    if (bf16) launch_few<kLinear, uint16_t>(p, plan, stream);
    else launch_few<kLinear, float>(p, plan, stream);
  } else {
    if (bf16) launch_many<kLinear, uint16_t>(p, plan, stream);
    else launch_many<kLinear, float>(p, plan, stream);
  }
  return hipGetLastError();
}

size_t ffn_i8_workspace_bytes(int n_rows, int n_tokens, int d, int I) {
  return ffn_i8_layout(n_rows, n_tokens, d, I).total;
}

hipError_t launch_ffn_i8(const FfnI8Args& a, void* workspace, hipStream_t stream) {
  char* ws = static_cast<char*>(workspace);
  const FfnI8Layout L = ffn_i8_layout(a.g.n_rows, a.g.n_x, a.d, a.I);
  if (few(a.g.n_rows, a.I)) {
    ProductArgs p = product_args(a.g, a.d, a.I);
    p.x = a.x;
    p.w0 = a.w_gate;
    p.w1 = a.w_up;
    p.s0 = a.s_gate;
    p.s1 = a.s_up;
    p.out = ws + L.aq;
    launch_few<kGateUp, float>(p, plan_ffn(kGateUp, sizes_of(p)), stream);
    ProductArgs h = product_args(a.g, a.I, a.d);
    h.af = reinterpret_cast<const float*>(ws + L.aq);
    h.w0 = a.w_down;
    h.s0 = a.s_down;
    h.out = a.h_sorted;
    launch_few<kDown, uint16_t>(h, plan_ffn(kDown, sizes_of(h)), stream);
    return hipGetLastError();
  }
  int8_t* xq = reinterpret_cast<int8_t*>(ws);
  float* xs = reinterpret_cast<float*>(ws + L.xs);
  const hipError_t e = launch_quantize_rows(a.x, 1, a.g.n_x, a.d, xq, xs, stream);
  if (e != hipSuccess) return e;
  ProductArgs p = product_args(a.g, a.d, a.I);
  p.a = xq;
  p.as = xs;
  p.w0 = a.w_gate;
  p.w1 = a.w_up;
  p.s0 = a.s_gate;
  p.s1 = a.s_up;
  p.out = ws + L.aq;
  p.out_scale = reinterpret_cast<float*>(ws + L.as);
  launch_many<kGateUp, int8_t>(p, plan_ffn(kGateUp, sizes_of(p)), stream);
  ProductArgs h = product_args(a.g, a.I, a.d);
  h.x_rows = nullptr;                       // the SwiGLU product is in sorted order
  h.n_x = a.g.n_rows;
  h.a = reinterpret_cast<const int8_t*>(ws + L.aq);
  h.as = p.out_scale;
  h.w0 = a.w_down;
  h.s0 = a.s_down;
  h.out = a.h_sorted;
  launch_many<kDown, uint16_t>(h, plan_ffn(kDown, sizes_of(h)), stream);
  return hipGetLastError();
}

}  // namespace moe
