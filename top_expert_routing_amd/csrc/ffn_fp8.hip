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
#include "fp8_plan.h"
#include "launch.h"
#include "tile_util.h"

namespace moe {

namespace {

using namespace fp8;

typedef int i32x8 __attribute__((ext_vector_type(8)));

static_assert(kBlock == kFp8Block && i8::kLanes == kWave, "one block size, one wavefront");
constexpr int kMaxGroups = 2 * 512 + 256;

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

// The same on the FP8 instructions: w and x are the two 16-byte pieces of each lane's columns.
__device__ __forceinline__ f32x4 mfma_codes(const uint4 (&w)[2], const uint4 (&x)[2]) {
  struct Two { uint4 v[2]; };
  const i32x8 a = __builtin_bit_cast(i32x8, (Two{{w[0], w[1]}}));
  const i32x8 b = __builtin_bit_cast(i32x8, (Two{{x[0], x[1]}}));
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
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

// ---- large groups: LDS-tiled products ----------------------------------------------
// A persistent block (one per CU) walks its list of tiles: BM rows x BN weight rows
// (kGateUp: 128 gate and the same 128 up rows).  K advances 128 codes a stage through a
// ring of LDS stages that LDS-DMA loads fill ahead; the stages of all tiles form one
// stream, so the next tile's first stages load while this one finishes.
//   * rows: a stage holds them as two halves of 64 codes, four 16-byte pieces each; piece c of row
//     r lies at slot c ^ swz(r), so that the 16 rows of an operand read hit different banks.  A DMA
//     instruction fills 16 rows (lane -> row lane / 4, slot lane % 4).
//   * weights: a packed block (16 rows x 64 codes, 1 KiB) is copied as it is.
//   * scales: one 4-byte load per wave and stage, its rows' in lanes 0 - 31, the matrix's (kGateUp:
//     gate's and up's, else those of the tile's two blocks of 128 columns) in lanes 32 and 33.
//   * the row list comes by DMA too, a tile ahead, because a load that the compiler sees would
//     make it wait for everything in flight.
// Waves: WM x WN, each MI x NJ blocks of 16x16; the 16-row blocks of the waves interleave, so the
// rows of a partial tile spread over them.
__device__ __forceinline__ int swz(int r) { return ((r >> 1) ^ (r >> 2)) & 3; }

template <class C, Mode M, bool EXACT, class Out>
__global__ __launch_bounds__(C::NT, C::NW / 4) void tile_fp8(ProductArgs p) {
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
  const int nb = (K + kBlock - 1) / kBlock, ncb = (cols + kBlock - 1) / kBlock;

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

  // ---- the loads, STAGES - 1 stages ahead of the products
  const uint32_t lds0 = lds_address(lds);
  const int halves = K / kHalf;
  uint32_t ao[C::ADMA], ao_next[C::ADMA];                      // this lane's bytes from p.a: tile being loaded, tile after it
  const uint8_t *bp[C::BDMA], *bp_next[C::BDMA];               // wave-uniform
  const float *sp, *sp_next;                                   // this lane's scales, one per stage, sstep apart
  // lane 16 i + r of a wave has row r of the 16 rows of its load i, so wave w's rows are the w-th 16 * ADMA of ROWS
  const bool vlane = lane < 16 * C::ADMA, slane = vlane || (lane >> 1) == 16;
  const int vrow = 16 * (wave + NW * (lane >> 4)) + l16;
  const size_t sstep = lane < 32 ? p.as_block : 1;
  auto load_list = [&](const Item& it, int parity) MOE_INLINE {
    if (p.x_rows && vlane)
      dma4(p.x_rows + it.row(min(vrow, it.rows - 1)), lds0 + L::LIST + parity * L::ROWS + wave * L::WROWS);
  };
  // Sources of a tile whose row list has arrived.
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
    const int second = lane & 1;
    const int cb = M == kGateUp ? it.chunk : min(it.chunk * (OUTC / kBlock) + second, ncb - 1);
    const float* sw = (M == kGateUp && second ? p.s1 : p.s0) + (static_cast<size_t>(it.expert) * ncb + cb) * nb;
    sp_next = vlane ? p.as + src(vrow, lane & (16 * C::ADMA - 1)) * p.as_row : sw;
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
  constexpr int CODES = 2 * (C::ADMA + C::BDMA);               // loads of a stage per wave: of codes,
  constexpr int PER = CODES + 1;                               // and one of scales
  auto load = [&](int i) MOE_INLINE {                          // the i-th of them
    const uint32_t st = lds0 + islot * L::STAGE;
    if (i == CODES) {
      if (slane) dma4(sp + ikt * sstep, st + 2 * (L::A + L::B) + wave * L::WSCALES);
      return;
    }
    const int h = i / (C::ADMA + C::BDMA), n = i % (C::ADMA + C::BDMA);
    const int kt = min(2 * ikt + h, halves - 1);               // the half past K: the last one again (see a1 below)
    if (n < C::ADMA) dma16(p.a + kt * kHalf, ao[n], st + h * L::A + (n * NW + wave) * 1024);
    else dma16(bp[n - C::ADMA] + static_cast<size_t>(kt) * 1024, lane * 16,
               st + 2 * L::A + h * L::B + ((n - C::ADMA) * NW + wave) * 1024);
  };
  auto loaded = [&]() MOE_INLINE {
    islot = islot + 1 == L::STAGES ? 0 : islot + 1;
    if (++ikt == nb) turn();
  };
  Item cur = item_of(0), nxt = n_my > 1 ? item_of(1) : cur;
  load_list(cur, 0);
  load_list(nxt, 1);
  wait_loads_barrier<0>();
  aim(cur, 0);
  turn();
#pragma unroll 1
  for (int s = 0; s < L::AHEAD; ++s) {                         // nb > AHEAD (kTileMinStages)
#pragma unroll
    for (int i = 0; i < PER; ++i) load(i);
    loaded();
  }

  // ---- compute side
  const int aoff = 16 * wm * kHalf + l16 * kHalf + 16 * (q ^ swz(l16));   // 16-row blocks do not change swz
  int cslot = 0;
  auto next_stage = [&]() MOE_INLINE {
    const uint8_t* st = lds + cslot * L::STAGE;
    cslot = cslot + 1 == L::STAGES ? 0 : cslot + 1;
    return st;
  };
  auto bfrag = [&](const uint8_t* st, int h, int j) MOE_INLINE {
    const int b = M == kGateUp ? (j < NJ / 2 ? wn * (NJ / 2) + j : C::BN / 32 + wn * (NJ / 2) + j - NJ / 2) : wn * NJ + j;
    return *reinterpret_cast<const uint4*>(st + 2 * L::A + h * L::B + b * 1024 + lane * 16);
  };
  auto afrag = [&](const uint8_t* st, int h, int i) MOE_INLINE {
    return *reinterpret_cast<const uint4*>(st + h * L::A + aoff + 16 * WM * i * kHalf);
  };
#pragma unroll 1
  for (int cr = 0; cr < n_my; ++cr) {
    const Item it = cur;
    const int par = cr & 1;
    // every wave is done with tile cr - 1: its list makes room for tile cr + 1's
    lds_barrier();
    aim(nxt, par ^ 1);
    cur = nxt;
    if (cr + 2 < n_my) nxt = item_of(cr + 2);
    load_list(nxt, par);
    f32x4 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int blocks = (it.rows + 15) >> 4;                    // 16-row blocks with rows
    const int nv = __builtin_amdgcn_readfirstlane(min(MI, max(0, (blocks - wm + WM - 1) / WM)));   // of them this wave's
    // the K loop over the first NI of the wave's 16-row blocks (one copy for each: a partial tile
    // skips its empty blocks' products and their scaling)
    auto run = [&](auto ni) MOE_INLINE {
      constexpr int NI = decltype(ni)::value;
#pragma unroll 1
      for (int kt = 0; kt < nb; ++kt) {
        wait_loads_barrier<(L::AHEAD - 1) * PER>();            // this stage is complete, every wave is past the last one
#pragma unroll
        for (int i = 0; i < PER; ++i) load(i);
        loaded();
        const uint8_t* st = next_stage();
        if constexpr (NI > 0) {
          // Past K both halves hold the same columns; the rows' second one counts as zeros.  (The weights'
          // may be NaN, but then so is the first half, which the row multiplies too.)
          const bool two = 2 * kt + 1 < halves;
          const float* sc = reinterpret_cast<const float*>(st + 2 * (L::A + L::B));
          const float* sw = sc + wave * (L::WSCALES / 4) + 32;
          const float w0 = sw[M == kGateUp || C::BN == kBlock ? 0 : wn], w1 = M == kGateUp ? sw[1] : w0;
          uint4 a[NI][2];
          float s[NI][2];
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            a[i][0] = afrag(st, 0, i);
            a[i][1] = two ? afrag(st, 1, i) : make_uint4(0, 0, 0, 0);
            const int blk = wm + WM * i;
            const float sx = sc[(blk % NW) * (L::WSCALES / 4) + (blk / NW) * 16 + l16];
            s[i][0] = sx * w0;
            s[i][1] = sx * w1;
          }
          if constexpr (EXACT) {
            Wide x[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) x[i] = widen(a[i]);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const uint4 b[2] = {bfrag(st, 0, j), bfrag(st, 1, j)};
              const Wide w = widen(b);
#pragma unroll
              for (int i = 0; i < NI; ++i) {
                const f32x4 t = mfma_wide(w, x[i]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(t[r], s[i][0], acc[i][j][r]);
              }
            }
          } else {
            // the sums of column block j are scaled into acc while block j + 1 multiplies,
            // and the operands of block j + 2 are read
            uint4 b[2] = {bfrag(st, 0, 0), bfrag(st, 1, 0)}, d[2] = {bfrag(st, 0, 1), bfrag(st, 1, 1)};
            f32x4 t[2][NI];
#pragma unroll
            for (int j = 0; j <= NJ; ++j) {
              uint4 c[2];
              if (j + 2 < NJ) c[0] = bfrag(st, 0, j + 2), c[1] = bfrag(st, 1, j + 2);
              if (j < NJ) {
#pragma unroll
                for (int i = 0; i < NI; ++i) t[j & 1][i] = mfma_codes(b, a[i]);
              }
              if (j > 0) {
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                  for (int r = 0; r < 4; ++r)
                    acc[i][j - 1][r] = __builtin_fmaf(t[(j - 1) & 1][i][r], s[i][M == kGateUp && j > NJ / 2 ? 1 : 0], acc[i][j - 1][r]);
              }
              if (j > 0 && j < NJ) {
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // the reads first, then one product, four sums, ...
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                  __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                  __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
                }
              }
              __builtin_amdgcn_sched_barrier(0);
              b[0] = d[0], b[1] = d[1], d[0] = c[0], d[1] = c[1];
            }
          }
        }
      }
    };
    static_assert(MI == 4 || MI == 2, "one copy for each number of blocks");
    if constexpr (MI == 4) {
      if (nv == 4) run(std::integral_constant<int, 4>{});
      else if (nv == 3) run(std::integral_constant<int, 3>{});
    }
    if (nv == 2) run(std::integral_constant<int, 2>{});
    else if (nv == 1) run(std::integral_constant<int, 1>{});
    else if (nv == 0) run(std::integral_constant<int, 0>{});

    // ---- epilogue
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
        static_assert(NJ / 2 == 4, "one 16-byte store per row and lane");
        uint32_t d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = block_codes(v[i][j], qs.r);
        transpose_rows(d);                                     // now lane 16 q + r: the 16 columns of block q
        if (m >= it.rows) continue;
        const int row = it.row(m), n = n0 + 16 * (wn * 4 + q);
        if (wn == 0 && q == 0) p.out_scale[static_cast<size_t>(it.chunk) * p.n_rows + row] = qs.base;
        if (n < cols)
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + static_cast<size_t>(row) * cols + n) =
              make_uint4(d[0], d[1], d[2], d[3]);
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
  // the stages requested past the last tile land in LDS: not after this block has left it
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <class Tile, Mode M, bool EXACT, class Out>
void launch_tile(const ProductArgs& p, hipStream_t stream) {
  const int cus = (device_cus() + kXcds - 1) / kXcds * kXcds;
  const size_t lds = TileLds<Tile, M>::bytes(p.G);
  hipLaunchKernelGGL((tile_fp8<Tile, M, EXACT, Out>), dim3(cus), dim3(Tile::NT), lds, stream, p);
}

Sizes sizes_of(const ProductArgs& p) { return Sizes{p.n_rows, p.E, p.G - p.nseg * p.E, p.nseg, p.K, p.cols}; }

template <Mode M, class Out>
void launch_product(const ProductArgs& p, hipStream_t stream) {
  constexpr bool exact = sizeof(Out) == 4;
  const Plan plan = fp8::plan(M, exact, sizes_of(p));
  if (plan.kernel == Kernel::kStream) {
    const Launch l = launch_of(i8::Plan{i8::Kernel::kStream, plan.width, plan.blocks});
    const dim3 grid(l.x, l.y), block(kThreadsS);
    if (plan.width == 1) hipLaunchKernelGGL((stream_fp8<1, M, Out>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((stream_fp8<2, M, Out>), grid, block, 0, stream, p);
  } else if constexpr (exact) {
    launch_tile<TileExact, M, true, Out>(p, stream);
  } else {
    if (plan.kernel == Kernel::kTileWide) launch_tile<TileWide, M, false, Out>(p, stream);
    else launch_tile<TileLow, M, false, Out>(p, stream);
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
