// Grouped products of block-scaled E4M3 rows and matrices (moe_grouped_linear_fp8,
// moe_grouped_ffn_fp8) on the matrix instructions of gfx950.
//
// Three kinds of products:
//   kLinear  y = sum over blocks b: sx[b] sw[b] * (xq . W over b)          -> bf16 or fp32
//   kGateUp  a = silu(x . Wg) * (x . Wu), coded per row and 128 columns (the columns of
//            one tile)                                                     -> codes + scales
//   kDown    kLinear on those codes                                        -> bf16
// A block's sum starts at zero in the matrix instructions, and one fma with sx * sw adds it to the
// running fp32 sum.
//
// The FP8 matrix instructions do not add in fp32: of each 8 columns of K they cut every product to a multiple of
// 2^(e - 13), e the exponent of the largest of the eight (measured: 1.5e-5 to 5e-5 of a sum in the 2-norm).
// tile_fp8 uses them where the result itself is rounded to bf16 (2^-9 of a value and more), at twice the rate.  Where it
// stays fp32, as for the gate and up sums, whose SwiGLU product is coded (cut sums turn one code of 650 into another one),
// and in the kernels of fewer rows, which wait for memory, the codes are widened to bf16, which has every E4M3 value,
// and multiplied by v_mfma_f32_16x16x32_bf16.
//
// Which of the 128 columns a lane holds does not matter as long as both operands agree:
// lane 16 q + r holds columns 16 q .. 16 q + 15 and 64 + 16 q .. 64 + 16 q + 15 of row r, which
// are 16 bytes of each of two packed KiB.  The weight rows are the first operand, so in a
// 16x16 result lane 16 q + r has token row r and the output columns 4 q .. 4 q + 3.
#include <type_traits>

#include "common.h"
#include "fp8_block.h"
#include "fp8_plan.h"
#include "launch.h"
#include "tile_util.h"

namespace moe {

namespace {

using namespace fp8;

typedef int i32x8 __attribute__((ext_vector_type(8)));

static_assert(kBlock == kFp8Block && i8::kLanes == kWave, "one block size, one wavefront");

struct ProductArgs {
  const uint8_t* a;        // codes of the rows: [n_x][K]
  const float* af;         // few_fp8<kDown>: the SwiGLU product [n_rows][K], in place of a and as
  const float* as;         // their scales: row r, block b at r * as_row + b * as_block
  size_t as_row, as_block;
  const uint8_t *w0, *w1;  // packed matrices [E+S][cols][K] (w1: up rows of kGateUp)
  const float *s0, *s1;    // their scales [E+S][ceil(cols / 128)][ceil(K / 128)]
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

// Half of a lane's columns as bf16, which has every E4M3 value.
struct Wide {
  bf16x8 v[4];
};
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ Wide widen(const uint4 (&c)[2]) {
  return Wide{{widen8(c[0].x, c[0].y), widen8(c[0].z, c[0].w), widen8(c[1].x, c[1].y), widen8(c[1].z, c[1].w)}};
}

// One block's sum: w and x are the lanes' columns of it.
__device__ __forceinline__ f32x4 mfma_wide(const Wide& w, const Wide& x) {
  f32x4 t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 4; ++h) t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[h], x.v[h], t, 0, 0, 0);
  return t;
}

// The same on the FP8 instructions: w and x are the two 16-byte pieces of each lane's columns.
__device__ __forceinline__ f32x4 mfma_codes(const uint4 (&w)[2], const uint4 (&x)[2]) {
  struct Two { uint4 v[2]; };
  const i32x8 a = __builtin_bit_cast(i32x8, (Two{{w[0], w[1]}}));
  const i32x8 b = __builtin_bit_cast(i32x8, (Two{{x[0], x[1]}}));
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// Codes of the SwiGLU product from v * (1 / scale) without the exact quotient's correction: v carries
// larger errors (fp32 sums, silu_mul), so a code may be the neighbour next to a border anyhow (measured: one of 2e5).
__device__ __forceinline__ Fp8Scale block_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return Fp8Scale{__builtin_nanf(""), 0.f};
  const float s = __uint_as_float(amax_bits) * (1.0f / 448.0f);
  if (s < 0x1p-100f) return Fp8Scale{1.f, 1.f};
  return Fp8Scale{s, __builtin_amdgcn_rcpf(s)};
}
__device__ __forceinline__ uint32_t block_codes(const float (&v)[4], float r) {
  if (r == 0.f) return 0;                                   // not finite: 0 * inf is no code
  return fp8_codes4(v[0] * r, v[1] * r, v[2] * r, v[3] * r);
}

// ---- small groups: weights stream from HBM into the matrix operands ----------------
// One block of eight waves per item (at most 16 * MF rows of a group, 128 output
// columns): each wave owns 16 columns (kGateUp: 16 gate rows and 16 up rows) and
// reads their weights once; the rows' codes are staged through LDS, 512 of K at a
// time (256 where two row blocks and two weight blocks fill the registers), double buffered,
// and shared by the waves.  Widening the codes is hidden by the weights' arrival.
// Bound by HBM: 128 tokens x 8 of 64 experts, 2048 -> 1408, 40 us for 190 MB (4.7 TB/s; a copy runs at 4.9).
constexpr int kThreadsS = 512;
constexpr int kWavesS = kThreadsS / kWave;

template <int MF, Mode M, class Out>
__global__ __launch_bounds__(kThreadsS, 4) void stream_fp8(ProductArgs p) {
  constexpr int BM = 16 * MF;
  constexpr int NF = M == kGateUp ? 2 : 1;
  constexpr int kChunk = NF * MF == 4 ? 256 : 512;
  constexpr int kPitch = kChunk + 16;                       // bytes of a staged row: 16 rows start in 16 different bank groups
  constexpr int BPC = kChunk / kBlock;                      // blocks of 128 in a chunk
  constexpr int VPR = kChunk / 16;                          // 16-byte pieces of a staged row
  constexpr int APT = BM * VPR / kThreadsS;                 // pieces per thread
  static_assert(BM * VPR % kThreadsS == 0, "whole pieces per thread");
  __shared__ __attribute__((aligned(16))) uint8_t As[2][BM * kPitch];
  __shared__ float Ss[2][BPC * BM];
  __shared__ uint32_t amax[M == kGateUp ? kWavesS : 1][M == kGateUp ? BM : 1];

  const int nch = (p.cols + kBlock - 1) / kBlock;
  const Item it = find_item(p, BM, nch);
  if (it.rows == 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  const int l16 = lane & 15, q = lane >> 4;
  const int K = p.K, cols = p.cols, nb = (K + kBlock - 1) / kBlock;
  const int col0 = it.chunk * kBlock + wave * 16;
  const bool live = col0 < cols;                            // cols % 64 == 0: all 16 columns or none
  const size_t rb = static_cast<size_t>(it.expert) * cols + (live ? col0 : cols - 16);
  const uint8_t* bp[NF];
  const float* sp[NF];                                      // the chunk's scales, one per block of K
  const size_t sb = (static_cast<size_t>(it.expert) * nch + it.chunk) * nb;
  bp[0] = p.w0 + rb * K + lane * 16;
  sp[0] = p.s0 + sb;
  if constexpr (NF == 2) bp[1] = p.w1 + rb * K + lane * 16, sp[1] = p.s1 + sb;

  const uint8_t* arow[APT];
  uint4 stage[APT];
  float sstage = 0.f;
#pragma unroll
  for (int s = 0; s < APT; ++s) {
    const int r = (threadIdx.x + s * kThreadsS) / VPR;
    arow[s] = r < it.rows ? p.a + static_cast<size_t>(src_row(p, it.row(r))) * K : nullptr;
  }
  const int sr = threadIdx.x % BM;                          // the row and block whose scale this thread stages
  const float* srow = threadIdx.x < BPC * BM && sr < it.rows
                          ? p.as + src_row(p, it.row(sr)) * p.as_row + threadIdx.x / BM * p.as_block : nullptr;
  auto load_a = [&](int c) MOE_INLINE {
#pragma unroll
    for (int s = 0; s < APT; ++s) {
      const int k = c * kChunk + (threadIdx.x + s * kThreadsS) % VPR * 16;
      stage[s] = arow[s] && k < K ? *reinterpret_cast<const uint4*>(arow[s] + k) : make_uint4(0, 0, 0, 0);
    }
    sstage = srow && c * BPC + static_cast<int>(threadIdx.x) / BM < nb ? srow[c * BPC * p.as_block] : 0.f;
  };
  auto store_a = [&](int buf) MOE_INLINE {
#pragma unroll
    for (int s = 0; s < APT; ++s) {
      const int i = threadIdx.x + s * kThreadsS;
      *reinterpret_cast<uint4*>(&As[buf][(i / VPR) * kPitch + (i % VPR) * 16]) = stage[s];
    }
    if (threadIdx.x < BPC * BM) Ss[buf][threadIdx.x] = sstage;
  };

  f32x4 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int nc = (K + kChunk - 1) / kChunk;
  load_a(0);
  store_a(0);
  for (int c = 0; c < nc; ++c) {
    uint4 b[BPC][NF][2];
    float sw[BPC][NF];
#pragma unroll
    for (int u = 0; u < BPC; ++u)
#pragma unroll
      for (int j = 0; j < NF; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int kk = c * kChunk + u * kBlock + h * kHalf;   // K % 64 == 0: whole halves; zeros past K on both sides
          b[u][j][h] = kk < K ? *reinterpret_cast<const uint4*>(bp[j] + static_cast<size_t>(kk) * 16) : make_uint4(0, 0, 0, 0);
        }
        sw[u][j] = sp[j][min(c * BPC + u, nb - 1)];
      }
    const bool more = c + 1 < nc;
    if (more) load_a(c + 1);
    __syncthreads();                                        // chunk c of the rows is staged
    const uint8_t* as = As[c & 1] + l16 * kPitch + 16 * q;
#pragma unroll
    for (int u = 0; u < BPC; ++u) {
      Wide w[NF];
#pragma unroll
      for (int j = 0; j < NF; ++j) w[j] = widen(b[u][j]);
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const uint4 av[2] = {*reinterpret_cast<const uint4*>(as + 16 * i * kPitch + u * kBlock),
                             *reinterpret_cast<const uint4*>(as + 16 * i * kPitch + u * kBlock + kHalf)};
        const Wide x = widen(av);
        const float sx = Ss[c & 1][u * BM + 16 * i + l16];
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const f32x4 t = mfma_wide(w[j], x);
          const float s = sx * sw[u][j];
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(t[r], s, acc[i][j][r]);
        }
      }
    }
    if (more) store_a((c + 1) & 1);                         // last read before this chunk's barrier
  }

  const int n = col0 + 4 * q;
  if constexpr (M == kGateUp) {
    float v[MF][4];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = 16 * i + l16;
      uint32_t big = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[i][r] = silu_mul(acc[i][0][r], acc[i][1][r]);
        big = max(big, abs_bits(v[i][r]));
      }
      big = max_over_q(big);
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
      const Fp8Scale qs = block_scale(big);
      const int row = it.row(m);
      if (live)
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + static_cast<size_t>(row) * cols + n) =
            block_codes(v[i], qs.r);
      if (wave == 0 && q == 0) p.out_scale[static_cast<size_t>(it.chunk) * p.n_rows + row] = qs.base;
    }
  } else {
    if (!live) return;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = 16 * i + l16;
      if (m >= it.rows) continue;
      const float v[4] = {acc[i][0][0], acc[i][0][1], acc[i][0][2], acc[i][0][3]};
      store4(static_cast<Out*>(p.out) + static_cast<size_t>(it.row(m)) * cols + n, v);
    }
  }
}

// ---- few rows: 16 columns per block, K split over its waves --------------------------
// With few rows (one token's experts, a small dense batch) 128-column items are too few
// to draw the weights through every CU, so an item is 16 columns (kGateUp: 16 gate and 16
// up rows; 32 or 64 where there are many) of at most 16 rows and the eight waves split K by
// whole blocks; their sums are joined through LDS in the order of the waves.
// A block does not hold the columns that share a scale of the SwiGLU product, so kGateUp writes
// that in fp32 (N * I * 4 bytes, at most 80 KiB here), and kDown's waves, each on whole blocks
// of 128 columns, quantise it as they read it.
// Bound by the latency of offsets, then rows and weights, then the join, around one burst: one token x 8 of 64 experts,
// 2048 x 1024, 9.5 + 6.6 us (33.8 and 17.2 MB); 5 rows x 2048 -> 2048 4.6 us (stream_fp8 8.5).
constexpr int kFewBlocksHeld = 2;        // blocks of K in flight per wave
constexpr int kSplit = kWavesS;

template <int NC, Mode M, class Out>
__global__ __launch_bounds__(kThreadsS, NC == 1 ? 4 : 2) void few_fp8(ProductArgs p) {
  constexpr int NF = M == kGateUp ? 2 * NC : NC, U = kFewBlocksHeld;   // j < NC: gate or only, j >= NC: up
  __shared__ f32x4 part[kSplit][NF][kWave];
  const Item it = find_item(p, 16, p.cols / (16 * NC));
  if (it.rows == 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  const int l16 = lane & 15, q = lane >> 4;
  const int K = p.K, cols = p.cols, nb = (K + kBlock - 1) / kBlock, ncb = (cols + kBlock - 1) / kBlock;
  // this wave's blocks of K, dealt in equal runs
  const int run = (nb + kSplit - 1) / kSplit;
  const int b0 = min(nb, wave * run), b1 = min(nb, b0 + run);
  const size_t rb = static_cast<size_t>(it.expert) * cols + it.chunk * 16 * NC;
  const size_t sb = (static_cast<size_t>(it.expert) * ncb + it.chunk * 16 * NC / kBlock) * nb;
  const uint8_t* wp[NF];                                    // wave-uniform; a lane's 16 bytes are its `lane`-th
#pragma unroll
  for (int j = 0; j < NF; ++j) wp[j] = (j < NC ? p.w0 : p.w1) + (rb + 16 * (j % NC)) * K;
  // Loads without branches, so that the waits count them one by one: a half past K loads the matrix's last
  // one (which its zeros of the rows multiply), a block past this wave's run what is not multiplied.
  auto half_at = [&](int b, int h) MOE_INLINE { return static_cast<size_t>(min(b * kBlock + h * kHalf, K - kHalf)); };
  uint4 w[U][NF][2];
  auto load_w = [&](int b, int u) MOE_INLINE {
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[u][j][h] = reinterpret_cast<const uint4*>(wp[j] + half_at(b + u, h) * 16)[lane];
  };
  // this lane's row (lanes past the rows repeat the last one) and its 32 columns of each block: codes, kDown fp32
  const int row = it.row(min(l16, it.rows - 1));
  constexpr int PIECES = M == kDown ? 8 : 2;
  uint4 x[U][PIECES];
  float sx[U], sw[U][2];
  const uint8_t* xr = nullptr;
  const float* sr = nullptr;
  auto load_x = [&](int b) MOE_INLINE {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int h = i / (PIECES / 2), k = i % (PIECES / 2);
        x[u][i] = reinterpret_cast<const uint4*>(xr + half_at(b + u, h) * (PIECES / 2))[k];
      }
      const int at = min(b + u, nb - 1);
      if constexpr (M != kDown) sx[u] = sr[at * p.as_block];
      sw[u][0] = p.s0[sb + at];
      if constexpr (M == kGateUp) sw[u][1] = p.s1[sb + at];
    }
  };
  // A wave's loads return in order, so the first rows are asked for among the first weights
  load_w(b0, 0);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (M == kDown) {
    xr = reinterpret_cast<const uint8_t*>(p.af + static_cast<size_t>(row) * K + 16 * q);
  } else {
    const int src = src_row(p, row);
    xr = p.a + static_cast<size_t>(src) * K + 16 * q;
    sr = p.as + src * p.as_row;
  }
  load_x(b0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int u = 1; u < U; ++u) load_w(b0, u);
  __builtin_amdgcn_sched_barrier(0);

  f32x4 acc[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int b = b0; b < b1; b += U) {
    if (b != b0) {
      load_x(b);
#pragma unroll
      for (int u = 0; u < U; ++u) load_w(b, u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u >= b1) break;
      const bool two = (b + u) * kBlock + kHalf < K;        // else the second half is past K: zeros
      uint4 c[2];
      if constexpr (M == kDown) {
        float v[8][4];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f32x4 f = __builtin_bit_cast(f32x4, x[u][i]);
          if (i >= 4 && !two) f = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            v[i][r] = f[r];
            m = max(m, abs_bits(f[r]));
          }
        }
        const Fp8Scale bs = block_scale(max_over_q(m));
        uint32_t d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = block_codes(v[i], bs.r);
        c[0] = make_uint4(d[0], d[1], d[2], d[3]);
        c[1] = make_uint4(d[4], d[5], d[6], d[7]);
        sx[u] = bs.base;
      } else {
        c[0] = x[u][0];
        c[1] = two ? x[u][1] : make_uint4(0, 0, 0, 0);
      }
      const Wide xw = widen(c);
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        const f32x4 t = mfma_wide(widen(w[u][j]), xw);
        const float s = sx[u] * sw[u][M == kGateUp && j >= NC ? 1 : 0];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][r] = __builtin_fmaf(t[r], s, acc[j][r]);
      }
    }
  }
  // join; wave j takes column block j
#pragma unroll
  for (int j = 0; j < NF; ++j) part[wave][j][lane] = acc[j];
  __syncthreads();
  if (wave >= NC || l16 >= it.rows) return;
  auto joined = [&](int j) MOE_INLINE {
    f32x4 v = part[0][j][lane];
#pragma unroll
    for (int i = 1; i < kSplit; ++i) v += part[i][j][lane];
    return v;
  };
  const int n = (it.chunk * NC + wave) * 16 + 4 * q;
  const f32x4 g = joined(wave);
  float v[4];
  if constexpr (M == kGateUp) {
    const f32x4 u = joined(NC + wave);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = silu_mul(g[r], u[r]);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = g[r];
  }
  store4(static_cast<Out*>(p.out) + static_cast<size_t>(row) * cols + n, v);
}

// ---- large groups: LDS-tiled products ----------------------------------------------
// A persistent block (one per CU) walks its list of tiles: BM rows x BN weight rows
// (kGateUp: 128 gate and the same 128 up rows).  K advances 128 codes a stage through a
// ring of LDS stages; the stages of all tiles form one stream, so the next tile's first
// stages load while this one finishes.
// Some waves multiply and four load.  A wave that requests an LDS-DMA load waits while the CU's address unit is
// busy, and it is busy most of the time: where all waves did both, a tile's time was the sum of the two (FFN of
// 96 rows for each of 64 experts, 2048 x 1024, 123 us with tiles of this size, 109 with waves that load; of 256 rows 238 / 191;
// 8192 rows x 8192 -> 4096 265 us with tiles of 256 x 256, 270 with these of 128 x 256).
// (FFN figures here and below compare two forms with both products on the FP8 instructions and 128 x 256 tiles.)
// What bounds it: at 8192 x 8192 -> 4096 the loads alone take 214 us (159 from a warm L2), the matrix instructions alone 134,
// those with their LDS reads 234.
// EXACT (fp32 out, and kGateUp) multiplies codes widened to bf16, at half the rate and with 16 conversions for each operand: four
// waves of 64 x 64, which share more of them than eight of 32 x 64 (8191 rows x 2048 -> 4096 166 us against 174, and 161 since
// the next tile is found early).  kGateUp's tile is 64 x 256, since it holds the columns of one scale twice, of gate and of up:
// FFN of 4096 tokens x 8 of 128 experts, 2048 x 768, 398 us, with eight waves of 32 x 64 405, on 128 x 256 with eight of 64 x 64,
// whose registers leave the widened operands no room to stay, 407; of 34 rows for each of 128 experts, 2880 x 2880, 613, 617, 850.
// (On the FP8 instructions, with cut sums, 298 and 618.)
//   * rows: 128 bytes of a row per stage, eight 16-byte pieces; piece c of row r lies at slot
//     c ^ ((r / 2) % 8), so that the 16 rows of an operand read hit different banks.  A DMA instruction
//     fills 8 rows (lane -> row lane / 8, slot lane % 8).
//   * weights: a packed block (16 rows x 64 codes, 1 KiB) is copied as it is.
//   * scales: those of four stages together, since a row's lie in one cache line: a 4-byte load for
//     each 16 rows (lane 4 r + k: row r, stage k), and one for the matrix's (kGateUp: gate's and up's,
//     else those of the tile's two blocks of 128 columns).
//   * the row list comes by DMA too, a tile ahead, because a load that the compiler sees would
//     make it wait for everything in flight.
// Barrier s, two passes before the end of step s (the multiplication of stage s), says that stage s + 1 has
// arrived and that stage s has been read: stage s + STAGES takes its place.
// Waves that multiply: WM x WN, each MI x NJ blocks of 16x16; the 16-row blocks of the waves interleave, so the
// rows of a partial tile spread over them.

// The lane's number, made anew: what is computed from it outside the K loop does not stay in registers through it.
__device__ __forceinline__ int fresh_lane() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(l));
  return l;
}

template <class C, Mode M, bool EXACT, class Out>
__global__ __launch_bounds__(C::NT, (C::NW + kLoaders) / 4) void tile_fp8(ProductArgs p) {
  using L = TileLds<C, M>;
  constexpr int MI = C::MI, NJ = C::NJ, WM = C::WM, WN = C::WN, NW = C::NW, NT = C::NT, BM = C::BM, STAGES = C::STAGES;
  constexpr int OUTC = M == kGateUp ? C::BN / 2 : C::BN;
  constexpr int GPT = (kTileMostGroups + NT - 1) / NT;
  constexpr int kPanel = 4;                                    // column chunks that follow each other per m-tile
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int* wsum = reinterpret_cast<int*>(lds + L::PLAN);
  int* before = wsum + NW + kLoaders;                          // m-tiles before group g
  int* offs = before + p.G + 1;
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = p.K, cols = p.cols;
  const int nb = (K + kBlock - 1) / kBlock, ncb = (cols + kBlock - 1) / kBlock, halves = K / kHalf;

  for (int g = tid; g <= p.G; g += NT) offs[g] = p.offs[g];
  if (tid < 4) reinterpret_cast<uint32_t*>(lds + L::ZERO)[tid] = 0;
  __syncthreads();
  {
    int cnt[GPT], sum = 0;
#pragma unroll
    for (int i = 0; i < GPT; ++i) {
      const int g = tid * GPT + i;
      cnt[i] = g < p.G ? group_rows(offs, p.n_rows, p.E, p.nseg, BM, g).nt : 0;
      sum += cnt[i];
    }
    const int incl = wave_prefix(sum);
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

  // ---- the waves that load ------------------------------------------------------------
  if (wave >= NW) {
    constexpr int AL = C::AL, BL = C::BL, SL = C::SL, PER = AL + 2 * BL;   // PER: loads of a stage's codes
    const int w = wave - NW;                                   // rows 8 AL w .., weight blocks BL w .. of a tile are this wave's
    const uint32_t lds0 = lds_address(lds);
    const uint32_t as_row = static_cast<uint32_t>(p.as_row), as_block = static_cast<uint32_t>(p.as_block);
    const uint32_t last = static_cast<uint32_t>(p.n_x) * K - 16;   // no row piece starts later: a short last stage's pieces past K
                                                               // are another row's, and not used (read_a)
    uint32_t ao[AL];                                           // of the tile being loaded: this lane's bytes from p.a,
    uint32_t so[SL];                                           // its rows' scales, in floats from p.as,
    const uint8_t* bp[BL];                                     // the weights (wave-uniform),
    const float *wp0, *wp1;                                    // the matrix's scales (wave-uniform)
    const uint32_t list0 = lds0 + L::LIST + w * 8 * AL * 4;
    auto load_list = [&](const Item& it, int parity) MOE_INLINE {
      if (p.x_rows && lane < 8 * AL)
        dma4(p.x_rows + it.row(min(8 * AL * w + lane, it.rows - 1)), list0 + parity * BM * 4);
    };
    // Sources of a tile whose row list has arrived.
    auto aim = [&](const Item& it, int parity) MOE_INLINE {
      const int* list = reinterpret_cast<const int*>(lds + L::LIST + (parity * BM + w * 8 * AL) * 4);
      auto src = [&](int r) MOE_INLINE {                       // of this wave's rows
        return p.x_rows ? min(max(list[r], 0), p.n_x - 1) : it.row(min(8 * AL * w + r, it.rows - 1));
      };
#pragma unroll
      for (int i = 0; i < AL; ++i) {
        const int r = 8 * i + (lane >> 3);
        ao[i] = static_cast<uint32_t>(src(r)) * K + 16 * ((lane & 7) ^ ((r >> 1) & 7));
      }
#pragma unroll
      for (int i = 0; i < SL; ++i) so[i] = src(16 * i + (lane >> 2)) * as_row + (lane & 3) * as_block;
      const int n0 = it.chunk * OUTC;
      const size_t e0 = static_cast<size_t>(it.expert) * cols;
#pragma unroll
      for (int i = 0; i < BL; ++i) {
        const int b = w * BL + i;                              // 16-row block of the tile
        const bool up = M == kGateUp && b >= C::BN / 32;
        const int n = min(n0 + 16 * (up ? b - C::BN / 32 : b), cols - 16);   // past the columns: read, never stored
        bp[i] = (up ? p.w1 : p.w0) + (e0 + n) * K;
      }
      const size_t sb = static_cast<size_t>(it.expert) * ncb;
      const int cb = M == kGateUp ? it.chunk : it.chunk * (OUTC / kBlock);
      wp0 = p.s0 + (sb + cb) * nb;
      wp1 = M == kGateUp ? p.s1 + (sb + cb) * nb : p.s0 + (sb + min(cb + 1, ncb - 1)) * nb;
    };
    // Part u of a group's scales: 16 of this wave's rows, or the matrix's; lanes past K's blocks take no part.
    auto load_scales = [&](int group, int slot, int u) MOE_INLINE {
      const int left = nb - group * kScaleGroup;
      const uint64_t four = left >= kScaleGroup ? 15 : left > 0 ? (1 << left) - 1 : 0;
      const uint32_t to = lds0 + L::SCALE0 + slot * L::SCALES;
      if (u < SL) {
        dma4(p.as, (so[SL > 1 && u == 1 ? SL - 1 : 0] + group * kScaleGroup * as_block) * 4, to + (w * SL + u) * 256,
             four * 0x1111111111111111ull);
      } else if (u == SL) {
        dma4((lane & 4 ? wp1 : wp0) + group * kScaleGroup + (lane & 3), to + L::WSCALE, w == 0 ? four * 0x11ull : 0);
      }
    };
    int tile = 0, ikt = 0, islot = 0, gslot = -1;              // the stage requested next: tile, number in it, ring slot; its group's slot
    Item next;                                                 // the tile after it
    auto look_ahead = [&](int t) MOE_INLINE {                  // written down for the waves that multiply
      next = item_of(t);
      if (w == 0 && lane == 0) *reinterpret_cast<Item*>(lds + L::ITEMS + t % kItemSlots * sizeof(Item)) = next;
      load_list(next, t & 1);
    };
    auto request = [&]() MOE_INLINE {
      // A group's scales are requested with the second and later stages of the group before, a tile's first group's with
      // its first stage.  At most two groups (three with four stages) lie between what is requested and what is read.
      auto after = [](int g) MOE_INLINE { return g + 1 == L::GROUPS ? 0 : g + 1; };
      const int u = ikt % kScaleGroup;
      if (u == 0) gslot = after(gslot);
      if (ikt == 0) {
#pragma unroll
        for (int i = 0; i <= SL; ++i) load_scales(0, gslot, i);
      } else if (u > 0) {
        load_scales(ikt / kScaleGroup + 1, after(gslot), u - 1);
      }
      const uint32_t to = lds0 + islot * L::STAGE, k = ikt * kBlock;
#pragma unroll
      for (int i = 0; i < AL; ++i) dma16(p.a + k, min(ao[i], last - k), to + (w * AL + i) * 1024);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int kt = min(2 * ikt + h, halves - 1);           // the half past K: the last one again (read_a)
#pragma unroll
        for (int i = 0; i < BL; ++i)
          dma16(bp[i] + static_cast<size_t>(kt) * 1024, lane * 16, to + L::A + h * L::B + (w * BL + i) * 1024);
      }
      islot = islot + 1 == STAGES ? 0 : islot + 1;
      // After a tile's last request the next one's sources, while this one's loads are on their way.  (Before its first
      // request, and with a search of their own by the waves that multiply: FFN of 4096 tokens x 8 of 128 experts, 2048 x 768,
      // 320 us instead of 290; of 1088 x 4 of 128, 2880 x 2880, 514 instead of 495.)
      if (++ikt == nb && tile + 1 < n_my) {
        if (nb < STAGES) wait_loads<0>();                      // its row list may be among the loads in flight
        ikt = 0;
        ++tile;
        aim(next, tile & 1);
        if (tile + 1 < n_my) look_ahead(tile + 1);
      }
    };
    look_ahead(0);
    const Item it0 = next;
    if (n_my > 1) look_ahead(1);
    wait_loads<0>();
    aim(it0, 0);
    const int total = n_my * nb;                               // at least kTileMinStages
    const int ahead = min(STAGES, total);
    for (int s = 0; s < ahead; ++s) request();
    if (ahead == STAGES) wait_loads<(STAGES - 1) * PER>();
    else wait_loads<0>();
    lds_barrier();                                             // stage 0 has arrived
    int to_end = nb;                                           // steps of the tile that is multiplied
    for (int s = 0; s < total; ++s) {
      if (s + STAGES <= total) wait_loads<(STAGES - 2) * PER>();
      else wait_loads<0>();
      lds_barrier();                                           // barrier s
      if (s + STAGES < total) request();
      if (--to_end == 0) {
        to_end = nb;
        if (M == kGateUp) barrier();                           // the epilogue's
      }
    }
    return;                                                    // nothing is in flight
  }

  // ---- the waves that multiply --------------------------------------------------------
  // A step goes through the wave's blocks by quarters, each a half of its row blocks with a half of its column
  // blocks, in an order in which neighbours share a half: rows 0 columns 0, rows 0 columns 1, rows 1 columns 1,
  // rows 1 columns 0.  A quarter of the operands is read during each quarter, into registers whose values are used up: this
  // step's columns 1 and rows 1, the next step's rows 0 and, each after its last use, columns 0.  (Rows all read in the
  // step's last quarter, 80 KiB for LDS within 256 cycles of matrix instructions: FFN of 4096 tokens x 8 of 128 experts,
  // 2048 x 768, 313 us instead of 297.  Columns alternating from step to step: two copies of the step, which spill.)
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t aoff = (16 * wm + (lane & 15)) * kBlock + 16 * ((lane >> 4) ^ ((lane & 15) >> 1));   // piece q; piece q + 4 is 64 bytes up or down
  uint4 fa[MI][2], fb[NJ][2];
  float sx[MI], sw[2];
  int cgroup = 0;                                              // slot of the scales that are read
  uint32_t cslot = 0, st = 0;                                  // the stage that is read: ring slot, place in LDS
  int ckt = 0;                                                 // its number in its tile
  auto at16 = [&](uint32_t a) MOE_INLINE { return *reinterpret_cast<const uint4*>(lds + a); };
  auto at4 = [&](uint32_t a) MOE_INLINE { return *reinterpret_cast<const float*>(lds + a); };
  auto read_a = [&](int i) MOE_INLINE {
    // Past K both halves hold the same columns; the rows' second one is read from zeros.  (The weights'
    // may be NaN, but then so is the first half, which the row multiplies too.)
    const uint32_t a = st + aoff;
    fa[i][0] = at16(a + 16 * WM * i * kBlock);
    fa[i][1] = at16(2 * ckt + 1 < halves ? (a ^ 64) + 16 * WM * i * kBlock : L::ZERO);
  };
  auto read_b = [&](int j) MOE_INLINE {
    const int b = M == kGateUp ? (j < NJ / 2 ? wn * (NJ / 2) + j : C::BN / 32 + wn * (NJ / 2) + j - NJ / 2) : wn * NJ + j;
#pragma unroll
    for (int h = 0; h < 2; ++h) fb[j][h] = at16(st + L::A + h * L::B + b * 1024 + lane * 16);
  };
  auto read_scales = [&]() MOE_INLINE {
    const uint32_t sc = L::SCALE0 + cgroup * L::SCALES + ckt % kScaleGroup * 4;
#pragma unroll
    for (int i = 0; i < MI; ++i) sx[i] = at4(sc + (16 * (wm + WM * i) + (lane & 15)) * 16);
    sw[0] = at4(sc + L::WSCALE + 16 * (M == kGateUp || C::BN == kBlock ? 0 : wn * NJ * 16 / kBlock));
    sw[1] = M == kGateUp ? at4(sc + L::WSCALE + 16) : sw[0];
  };
  barrier();                                                   // stage 0 has arrived
  read_scales();
  constexpr int HA = MI / 2, HB = NJ / 2, QUARTER = HA * HB;
#pragma unroll
  for (int i = 0; i < HA; ++i) read_a(i);
#pragma unroll
  for (int j = 0; j < HB; ++j) read_b(j);
#pragma unroll 1
  for (int cr = 0; cr < n_my; ++cr) {
    f32x4 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // A product is scaled into acc LAG products later; the step's last ones in the next step.
    constexpr int LAG = EXACT ? QUARTER : 3, RING = EXACT ? 2 * QUARTER : 4;
    static_assert(LAG <= QUARTER && 4 * QUARTER % RING == 0, "");
    f32x4 t[RING];
    float s[2][MI], s_last[MI];                                // rows' times gate's (the only), up's; of the step before
#pragma unroll
    for (int i = 0; i < RING; ++i) t[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < MI; ++i) s_last[i] = 0.f;
    // Row and column block of product n of a step's order, n < 0: of the step before.
    auto row_of = [](int n) MOE_INLINE { return (n < 0 || n >= 2 * QUARTER ? HA : 0) + (n + 4 * QUARTER) % HA; };
    auto col_of = [](int n) MOE_INLINE {
      const int quarter = (n + 4 * QUARTER) / QUARTER % 4;
      return (quarter == 1 || quarter == 2 ? HB : 0) + (n + 4 * QUARTER) % QUARTER / HA;
    };
    auto add = [&](int n) MOE_INLINE {
      const int i = row_of(n), j = col_of(n);
      const float by = n < 0 ? s_last[i] : s[M == kGateUp && j >= HB ? 1 : 0][i];
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(t[(n + 4 * QUARTER) % RING][r], by, acc[i][j][r]);
    };
#pragma unroll 1
    for (int kt = 0; kt < nb; ++kt) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        s[0][i] = sx[i] * sw[0];
        s[1][i] = sx[i] * sw[1];
      }
      Wide x[EXACT ? HA : 1], w[EXACT ? HB : 1];
#pragma unroll
      for (int quarter = 0; quarter < 4; ++quarter) {
        const int i0 = quarter < 2 ? 0 : HA, j0 = quarter == 1 || quarter == 2 ? HB : 0;
        if (quarter == 2) {
          lds_barrier();                                       // barrier of this step: this wave has read its stage
          cslot = cslot + 1 == STAGES ? 0 : cslot + 1;
          ckt = ckt + 1 == nb ? 0 : ckt + 1;
          st = cslot * L::STAGE;
          if (ckt % kScaleGroup == 0) cgroup = cgroup + 1 == L::GROUPS ? 0 : cgroup + 1;
        }
        if constexpr (EXACT) {
          if (quarter % 2 == 0) {
#pragma unroll
            for (int i = 0; i < HA; ++i) x[i] = widen(fa[i0 + i]);
          }
          if (quarter != 2) {
#pragma unroll
            for (int j = 0; j < HB; ++j) w[j] = widen(fb[j0 + j]);
          }
#pragma unroll
          for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int n = 0; n < QUARTER; ++n) {
              f32x4& to = t[(quarter * QUARTER + n) % RING];
              to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[EXACT ? n / HA : 0].v[h], x[EXACT ? n % HA : 0].v[h],
                                                           h ? to : f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
            }
        }
        // What is read now is used in the next quarter first (rows 0 in the one after).
#pragma unroll
        for (int n = 0; n < QUARTER; ++n) {
          const int m = quarter * QUARTER + n;
          if constexpr (!EXACT) t[m % RING] = mfma_codes(fb[j0 + n / HA], fa[i0 + n % HA]);
          const int u = n / HA;                                // a read per operand
          if (quarter == 0 && n % HA == 0) read_b(HB + u);
          if (quarter == 1 && n < HA) read_a(HA + n);
          if (quarter == 2 && n < HA) read_a(n);
          if (quarter == 3 && n % HA == HA - 1) read_b(u);
          if (quarter == 2 && n == QUARTER - 1) read_scales();
          add(m - LAG);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = HA; i < MI; ++i) s_last[i] = s[0][i];
    }
#pragma unroll
    for (int n = -LAG; n < 0; ++n) add(n);

    // ---- epilogue
    const Item it = uniform(*reinterpret_cast<const Item*>(lds + L::ITEMS + cr % kItemSlots * sizeof(Item)));
    const int elane = fresh_lane(), l16 = elane & 15, q = elane >> 4;
    const int n0 = it.chunk * OUTC;
    if constexpr (M == kGateUp) {
      uint32_t* mx = reinterpret_cast<uint32_t*>(lds + L::MAX);
      float v[MI][NJ / 2][4];
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int blk = wm + WM * i;
        uint32_t big = 0;
#pragma unroll
        for (int j = 0; j < NJ / 2; ++j) {
          const int c = 16 * (wn * (NJ / 2) + j) + 4 * q;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            v[i][j][r] = silu_mul(acc[i][j][r], acc[i][NJ / 2 + j][r]);
            if (n0 + c < cols) big = max(big, abs_bits(v[i][j][r]));
          }
        }
        big = max_over_q(big);
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
        const Fp8Scale qs = block_scale(big);
        uint32_t d[NJ / 2];
#pragma unroll
        for (int j = 0; j < NJ / 2; ++j) d[j] = block_codes(v[i][j], qs.r);
        const int row = it.row(min(m, it.rows - 1));
        uint8_t* orow = static_cast<uint8_t*>(p.out) + static_cast<size_t>(row) * cols;
        if (m < it.rows && wn == 0 && q == 0) p.out_scale[static_cast<size_t>(it.chunk) * p.n_rows + row] = qs.base;
        static_assert(NJ / 2 == 2, "one store per row and lane");
        swap32(d[0], d[1]);                                  // row q = 2 a + b gets columns 8 b .. 8 b + 7 of block a
        swap16(d[0], d[1]);
        const int n = n0 + 16 * (wn * 2 + (q >> 1)) + 8 * (q & 1);
        if (m < it.rows && n < cols) *reinterpret_cast<uint2*>(orow + n) = make_uint2(d[0], d[1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int blk = wm + WM * i, m = 16 * blk + l16;
        if (16 * blk >= it.rows) continue;                     // wave-uniform
        const bool in = m < it.rows;
        Out* orow = static_cast<Out*>(p.out) + static_cast<size_t>(it.row(in ? m : 0)) * cols + n0;
        if constexpr (sizeof(Out) == 4) {
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const int c = 16 * (wn * NJ + j) + 4 * q;
            const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            if (in && n0 + c < cols) store4(orow + c, v);
          }
        } else {
          // bf16: two column blocks to 16 bytes a lane: row q = 2 a + b gets columns 8 b .. 8 b + 7 of block j + a
#pragma unroll
          for (int j = 0; j < NJ; j += 2) {
            const f32x4 v = acc[i][j], u = acc[i][j + 1];
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
}

template <class Tile, Mode M, bool EXACT, class Out>
void launch_tile(const ProductArgs& p, hipStream_t stream) {
  const int cus = (device_cus() + kXcds - 1) / kXcds * kXcds;
  const size_t lds = TileLds<Tile, M>::bytes(p.G);
  hipLaunchKernelGGL((tile_fp8<Tile, M, EXACT, Out>), dim3(cus), dim3(Tile::NT), lds, stream, p);
}

Sizes sizes_of(const ProductArgs& p) { return Sizes{p.n_rows, p.E, p.G - p.nseg * p.E, p.nseg, p.K, p.cols}; }

template <Mode M, class Out>
void launch_few(const ProductArgs& p, hipStream_t stream) {
  const Plan plan = few_plan(M, sizes_of(p));
  const Launch l = launch_of(plan);
  const dim3 grid(l.x, l.y), block(kThreadsS);
  if (plan.width == 1) hipLaunchKernelGGL((few_fp8<1, M, Out>), grid, block, 0, stream, p);
  else if (plan.width == 2) hipLaunchKernelGGL((few_fp8<2, M, Out>), grid, block, 0, stream, p);
  else if constexpr (M != kGateUp) hipLaunchKernelGGL((few_fp8<4, M, Out>), grid, block, 0, stream, p);
}

template <Mode M, class Out>
void launch_many(const ProductArgs& p, hipStream_t stream) {
  constexpr bool exact = sizeof(Out) == 4;
  const Plan plan = many_plan(M, exact, sizes_of(p));
  if (plan.kernel == Kernel::kStream) {
    const Launch l = launch_of(plan);
    const dim3 grid(l.x, l.y), block(kThreadsS);
    if (plan.width == 1) hipLaunchKernelGGL((stream_fp8<1, M, Out>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((stream_fp8<2, M, Out>), grid, block, 0, stream, p);
  } else if constexpr (exact) {
    launch_tile<TileExact, M, true, Out>(p, stream);
  } else if constexpr (M == kGateUp) {                       // its sums stay fp32 until they are coded
    launch_tile<TileGateUp, M, true, Out>(p, stream);
  } else {
    launch_tile<TileCodes, M, false, Out>(p, stream);
  }
}

ProductArgs product_args(const GroupedFp8& g, int K, int cols) {
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

// Workspace of the FFN: SwiGLU codes and block scales; of few rows, the product in fp32.
struct FfnFp8Layout {
  size_t as, total;   // byte offsets (the codes start at 0)
};
FfnFp8Layout ffn_fp8_layout(int n_rows, int I) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  FfnFp8Layout L;
  L.as = up(static_cast<size_t>(n_rows) * I * (few_ffn(n_rows, I) ? 4 : 1));
  L.total = L.as + up(static_cast<size_t>((I + kBlock - 1) / kBlock) * n_rows * 4);
  return L;
}

}  // namespace

hipError_t launch_grouped_linear_fp8(const GroupedFp8& g, const uint8_t* xq, const float* xs, int K, int O,
                                     const uint8_t* w, const float* ws, int bf16, void* y, hipStream_t stream) {
  ProductArgs p = product_args(g, K, O);
  p.a = xq;
  p.as = xs;
  p.as_row = (K + kBlock - 1) / kBlock;
  p.as_block = 1;
  p.w0 = w;
  p.s0 = ws;
  p.out = y;
  if (few_linear(sizes_of(p))) {
    if (bf16) launch_few<kLinear, uint16_t>(p, stream);
    else launch_few<kLinear, float>(p, stream);
  } else {
    if (bf16) launch_many<kLinear, uint16_t>(p, stream);
    else launch_many<kLinear, float>(p, stream);
  }
  return hipGetLastError();
}

size_t ffn_fp8_workspace_bytes(int n_rows, int I) { return ffn_fp8_layout(n_rows, I).total; }

hipError_t launch_ffn_fp8(const FfnFp8Args& a, void* workspace, hipStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const FfnFp8Layout L = ffn_fp8_layout(a.g.n_rows, a.I);
  ProductArgs p = product_args(a.g, a.d, a.I);
  p.a = a.xq;
  p.as = a.xs;
  p.as_row = (a.d + kBlock - 1) / kBlock;
  p.as_block = 1;
  p.w0 = a.w_gate;
  p.w1 = a.w_up;
  p.s0 = a.s_gate;
  p.s1 = a.s_up;
  p.out = ws;
  p.out_scale = reinterpret_cast<float*>(ws + L.as);
  const bool fp32 = few_ffn(a.g.n_rows, a.I);
  if (fp32) launch_few<kGateUp, float>(p, stream);
  else launch_many<kGateUp, uint8_t>(p, stream);
  ProductArgs h = product_args(a.g, a.I, a.d);
  h.x_rows = nullptr;                       // the SwiGLU product is in sorted order
  h.n_x = a.g.n_rows;
  h.a = ws;
  h.af = reinterpret_cast<const float*>(ws);
  h.as = p.out_scale;
  h.as_row = 1;
  h.as_block = a.g.n_rows;
  h.w0 = a.w_down;
  h.s0 = a.s_down;
  h.out = a.h_sorted;
  if (fp32) launch_few<kDown, uint16_t>(h, stream);
  else launch_many<kDown, uint16_t>(h, stream);
  return hipGetLastError();
}

}  // namespace moe
