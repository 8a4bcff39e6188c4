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
// The codes are widened to bf16, which has every E4M3 value, and multiplied by
// v_mfma_f32_16x16x32_bf16, because the FP8 matrix instructions do not add in fp32: of each 8 columns
// of K they cut every product to a multiple of 2^(e - 13), e the exponent of the largest of the eight
// (measured: 1.5e-5 to 5e-5 of a sum in the 2-norm).
//
// Which of the 128 columns a lane holds does not matter as long as both operands agree:
// lane 16 q + r holds columns 16 q .. 16 q + 15 and 64 + 16 q .. 64 + 16 q + 15 of row r, which
// are 16 bytes of each of two packed KiB.  The weight rows are the first operand, so in a
// 16x16 result lane 16 q + r has token row r and the output columns 4 q .. 4 q + 3.
#include <type_traits>

#include "common.h"
#include "fp8_block.h"
#include "i8_plan.h"
#include "launch.h"
#include "tile_util.h"

namespace moe {

namespace {

using i8::kDown;
using i8::kGateUp;
using i8::kLinear;
using i8::Mode;

constexpr int kBlock = kFp8Block;
constexpr int kHalf = 64;                // columns of a packed block: half of what an instruction takes

struct ProductArgs {
  const uint8_t* a;        // codes of the rows: [n_x][K]
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

// Codes of the SwiGLU product from v * (1 / scale) without the exact quotient's correction: the
// products carry larger errors (silu_mul), so a code may be the neighbour next to a border anyhow.
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
// and shared by the waves.
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

i8::Sizes sizes_of(const ProductArgs& p) { return i8::Sizes{p.n_rows, p.E, p.G - p.nseg * p.E, p.nseg, p.K, p.cols}; }

template <Mode M, class Out>
void launch_product(const ProductArgs& p, hipStream_t stream) {
  const i8::Sizes s = sizes_of(p);
  const int nch = (p.cols + kBlock - 1) / kBlock, mf = i8::pick_mf(s.n_rows / s.sequences());
  const i8::Launch l = i8::launch_of(i8::Plan{i8::Kernel::kStream, mf, item_grid(i8::max_m_tiles(s, 16 * mf), nch)});
  const dim3 grid(l.x, l.y), block(kThreadsS);
  if (mf == 1) hipLaunchKernelGGL((stream_fp8<1, M, Out>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((stream_fp8<2, M, Out>), grid, block, 0, stream, p);
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

// Workspace of the FFN: SwiGLU codes and block scales.
struct FfnFp8Layout {
  size_t as, total;   // byte offsets (the codes start at 0)
};
FfnFp8Layout ffn_fp8_layout(int n_rows, int I) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  FfnFp8Layout L;
  L.as = up(static_cast<size_t>(n_rows) * I);
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
  if (bf16) launch_product<kLinear, uint16_t>(p, stream);
  else launch_product<kLinear, float>(p, stream);
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
  launch_product<kGateUp, uint8_t>(p, stream);
  ProductArgs h = product_args(a.g, a.I, a.d);
  h.x_rows = nullptr;                       // the SwiGLU product is in sorted order
  h.n_x = a.g.n_rows;
  h.a = ws;
  h.as = p.out_scale;
  h.as_row = 1;
  h.as_block = a.g.n_rows;
  h.w0 = a.w_down;
  h.s0 = a.s_down;
  h.out = a.h_sorted;
  launch_product<kDown, uint16_t>(h, stream);
  return hipGetLastError();
}

}  // namespace moe
