// Which kernel runs a block-scaled FP8 product (ffn_fp8.hip) and how much LDS its tiles take, from the
// sizes alone: host arithmetic without GPU code, so that a host program can ask it too.
#pragma once

#include "i8_plan.h"

namespace moe {
namespace fp8 {

using i8::kDown;
using i8::kGateUp;
using i8::kLinear;
using i8::Launch;
using i8::max_m_tiles;
using i8::Mode;
using i8::Sizes;

constexpr int kBlock = 128;          // columns that share a scale, and K of a stage
constexpr int kHalf = 64;            // columns of a packed block

// ---- tile_fp8's tiles and their LDS ---------------------------------------------------
// MI x NJ blocks of 16x16 per wave, WM x WN waves.
template <int MI_, int NJ_, int WM_, int WN_>
struct TileCfg {
  static constexpr int MI = MI_, NJ = NJ_, WM = WM_, WN = WN_, NW = WM * WN, NT = i8::kLanes * NW;
  static constexpr int BM = 16 * MI * WM, BN = 16 * NJ * WN;
  static constexpr int ADMA = BM / 16 / NW, BDMA = BN / 16 / NW;   // a wave's 16-row blocks
  static_assert(ADMA >= 1 && ADMA < 4 && BDMA >= 1, "a load of scales per stage: each 16 rows', the matrix's");
};
using TileWide = TileCfg<4, 8, 4, 2>;    // 256 rows x 256 weight rows
using TileLow = TileCfg<4, 4, 2, 4>;     // 128 rows x 256
using TileExact = TileCfg<4, 4, 4, 2>;   // 256 rows x 128

constexpr int kTileMinStages = 3;        // fewest stages (blocks of K) of a tile (TileLds)
constexpr int kScaleGroup = 4;           // stages whose scales are loaded together
template <class C, Mode M>
struct TileLds {
  static constexpr int A = C::BM * kBlock, B = C::BN * kHalf;  // bytes of a stage's rows, of half a stage's weights
  static constexpr int STAGE = A + 2 * B;
  // scales of a group of stages: a wave's are its rows' (16 bytes each), then those of two blocks of the matrix
  static constexpr int WSCALES = (16 * C::ADMA + 2) * 4 * kScaleGroup, SCALES = C::NW * WSCALES, GROUPS = 3;
  static constexpr int WROWS = 16 * C::ADMA * 4, ROWS = C::NW * WROWS;
  static constexpr int FIXED = GROUPS * SCALES + 2 * ROWS + (M == kGateUp ? C::WN * C::BM * 4 : 0) + 16;
  static constexpr int plan_bytes(int G) { return 4 * C::NW + 8 * (G + 1); }
  static constexpr int kMostGroups = 2 * 512 + 256;
  static constexpr int STAGES = (i8::kLdsPerCu - FIXED - plan_bytes(kMostGroups)) / STAGE;
  static constexpr int AHEAD = STAGES;                         // stages requested before the first is multiplied
  static_assert(STAGES >= 2 && (M != kGateUp || C::BN == 2 * kBlock), "a kGateUp tile holds the columns of one scale");
  static constexpr int RING = STAGES * STAGE, PLAN_ = RING + FIXED;
  static constexpr int SCALE0 = RING;                          // scales of three groups of stages
  static constexpr int LIST = RING + GROUPS * SCALES;                            // row list of two tiles
  static constexpr int MAX = LIST + 2 * ROWS;                  // kGateUp: largest magnitudes
  static constexpr int ZERO = PLAN_ - 16;                      // zeros
  static constexpr int PLAN = PLAN_;                    // sums over waves, tiles before each group, group offsets
  static int bytes(int G) { return PLAN + plan_bytes(G); }
  // The stages requested before a block's first product are all its first tile's: what follows is
  // the next tile's, whose sources are set when the first tile starts.
  static_assert(AHEAD <= kTileMinStages, "a tile has more stages than are requested ahead");
};

enum class Kernel { kFew, kStream, kTileLow, kTileWide, kTileExact };
struct Plan {
  Kernel kernel;
  int width;    // few_fp8: 16-column blocks of an item; stream_fp8: 16-row blocks of a tile
  int blocks;   // few_fp8, stream_fp8: blocks of the launch (tile_fp8's walk a list)
};
inline Launch launch_of(const Plan& p) { return i8::launch_of(i8::Plan{i8::Kernel::kStream, p.width, p.blocks}); }

constexpr int kTileMinAvg = 64, kWideMinAvg = 192;
constexpr int kTileMinItems = 512;

// The FFN's products of few rows (both of them: the SwiGLU product is kept in fp32 then).
inline bool few_ffn(int n_rows, int I) { return i8::few(n_rows, I); }
inline bool few_linear(const Sizes& s) {
  return static_cast<long long>(max_m_tiles(s, 16)) * (s.cols / 16) <= i8::kFewBlocksMost;
}
inline Plan few_plan(Mode m, const Sizes& s) {
  const i8::Plan p = i8::plan_few(m, s);
  return Plan{Kernel::kFew, p.width, p.blocks};
}

// exact: fp32 out
inline Plan many_plan(Mode m, bool exact, const Sizes& s) {
  const int avg = s.n_rows / s.sequences();
  const long long area = static_cast<long long>(s.n_rows) * s.cols;
  if (avg > kTileMinAvg && area >= kTileMinItems * 64ll * 128 && s.K > (kTileMinStages - 1) * kBlock)
    return Plan{exact ? Kernel::kTileExact : avg >= kWideMinAvg ? Kernel::kTileWide : Kernel::kTileLow, 0, 0};
  const int nch = (s.cols + kBlock - 1) / kBlock, mf = i8::pick_mf(avg);
  return Plan{Kernel::kStream, mf, item_grid(max_m_tiles(s, 16 * mf), nch)};
}

inline Plan linear_plan(bool exact, const Sizes& s) { return few_linear(s) ? few_plan(kLinear, s) : many_plan(kLinear, exact, s); }

// kGateUp: K = d, cols = I; kDown: K = I, cols = d.
inline Plan ffn_plan(Mode m, const Sizes& s) {
  return few_ffn(s.n_rows, m == kGateUp ? s.cols : s.K) ? few_plan(m, s) : many_plan(m, false, s);
}

}  // namespace fp8
}  // namespace moe
