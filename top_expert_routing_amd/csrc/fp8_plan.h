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
// MI x NJ blocks of 16x16 per wave that multiplies, WM x WN of them, and waves that only load.
constexpr int kLoaders = 4;
template <int MI_, int NJ_, int WM_, int WN_, int STAGES_>
struct TileCfg {
  static constexpr int MI = MI_, NJ = NJ_, WM = WM_, WN = WN_, NW = WM * WN, NT = i8::kLanes * (NW + kLoaders);
  static constexpr int BM = 16 * MI * WM, BN = 16 * NJ * WN, STAGES = STAGES_;
  static constexpr int AL = BM / 8 / kLoaders;                 // DMA instructions of a stage per loader: of rows (8 each),
  static constexpr int BL = BN / 16 / kLoaders;                // of weights, 16-row blocks (two halves each)
  static constexpr int SL = BM / 16 / kLoaders;                // of scales, 16 rows each, for a group of stages
  static_assert(SL >= 1 && SL < 3 && BL >= 1, "a load of scales per stage, but the group's first: rows', the matrix's");
};
using TileCodes = TileCfg<4, 4, 2, 4, 3>;   // 128 rows x 256 weight rows
using TileExact = TileCfg<4, 4, 2, 2, 4>;   // 128 rows x 128
using TileGateUp = TileCfg<4, 4, 1, 4, 3>;  // 64 rows x 128 gate and the same 128 up rows

constexpr int kTileMinStages = 3;        // fewest stages (blocks of K) of a tile: a row list arrives within them (tile_fp8)
constexpr int kScaleGroup = 4;           // stages whose scales are loaded together
// A tile is written down when the one before it begins to be requested, and stages are requested at most STAGES steps before
// they are multiplied: by the time that a tile is stored, three later ones are written down with the shortest tiles.
constexpr int kItemSlots = 8;
template <class C, Mode M>
struct TileLds {
  static constexpr int A = C::BM * kBlock, B = C::BN * kHalf;  // bytes of a stage's rows, of half a stage's weights
  static constexpr int STAGE = A + 2 * B;
  static constexpr int WSCALE = C::BM * 4 * kScaleGroup;       // in a group of scales: the rows' (16 bytes each), then of two
  static constexpr int SCALES = WSCALE + 2 * 4 * kScaleGroup;  // blocks of the matrix
  static constexpr int GROUPS = C::STAGES;                     // (tile_fp8)
  static_assert(M != kGateUp || C::BN == 2 * kBlock, "a kGateUp tile holds the columns of one scale");
  static_assert(C::STAGES - 1 <= kTileMinStages, "a tile's row list arrives before its first stage is requested");
  static constexpr int SCALE0 = C::STAGES * STAGE;
  static constexpr int LIST = SCALE0 + GROUPS * SCALES;        // row lists of two tiles
  static constexpr int MAX = LIST + 2 * C::BM * 4;             // kGateUp: largest magnitudes
  static constexpr int ZERO = MAX + (M == kGateUp ? C::WN * C::BM * 4 : 0);
  static constexpr int ITEMS = ZERO + 16;                      // the tiles that are loaded and multiplied
  static constexpr int PLAN = ITEMS + kItemSlots * static_cast<int>(sizeof(Item));                        // sums over waves, tiles before each group, group offsets
  static constexpr int bytes(int G) { return PLAN + 4 * (C::NW + kLoaders) + 8 * (G + 1); }
};
constexpr int kTileMostGroups = 800;     // whose lists fit beside the stages
static_assert(TileLds<TileCodes, kLinear>::bytes(kTileMostGroups) <= i8::kLdsPerCu &&
              TileLds<TileGateUp, kGateUp>::bytes(kTileMostGroups) <= i8::kLdsPerCu &&
              TileLds<TileExact, kLinear>::bytes(kTileMostGroups) <= i8::kLdsPerCu, "a block's LDS");

// kTile: results of 16 bits or fewer (TileCodes; kGateUp: TileGateUp), kTileExact: fp32 results
enum class Kernel { kFew, kStream, kTile, kTileExact };
struct Plan {
  Kernel kernel;
  int width;    // few_fp8: 16-column blocks of an item; stream_fp8: 16-row blocks of a tile
  int blocks;   // few_fp8, stream_fp8: blocks of the launch (tile_fp8's walk a list)
};
inline Launch launch_of(const Plan& p) { return i8::launch_of(i8::Plan{i8::Kernel::kStream, p.width, p.blocks}); }

// Where tile_fp8 takes over from stream_fp8: few rows per group leave its tiles of 128 (gate/up: 64) empty, and a small output
// leaves CUs without one, each of them as long as K.  us, stream_fp8 / tile_fp8 (products alone of 2^20 outputs, FFNs of groups):
//   outputs  linear 2048 -> 2048, 1024 rows (2.0) 21.1 / 22.0, 1536 rows (3.0) 28.9 / 22.7; 1024 -> 512, 2048 rows (1.0)
//            13.8 / 14.9, 3000 rows (1.5) 19.1 / 15.1; 2560 -> 2560, 512 rows (1.3) 23.2 / 24.7, 768 rows (1.9) 31.4 / 25.1;
//            fp32 out: 2048 -> 2048, 1536 rows 28.6 / 25.8; 1024 -> 512, 2048 rows 14.4 / 16.0
//   rows     where every group's one tile makes kTileManyItems (three a CU), fewer rows are enough: groups' sizes even / falling
//            as 1 / rank: FFN of 128 groups, 2880 x 2880, 16 rows 560 / 589 and 400 / 376, 20 rows 564 / 593 and 450 / 414, 28 rows
//            597 / 600 and 536 / 481, 34 rows 692 / 606 and 600 / 527; 128 groups, 2048 x 768, 20 rows 143 / 139 and 124 / 119, 28
//            rows 148 / 142 and 147 / 136; else: 64 groups, 2048 x 1024, 34 rows 105 / 104 and 104 / 115, 48 rows 111 / 108 and
//            118 / 117; 32 groups, 2880 x 2880, 28 rows 179 / 177 and 190 / 193, 39 rows 215 / 184 and 218 / 206
//            fp32 out: 64 groups 2048 -> 1024, 48 rows 40.3 / 43.1, 64 rows 46.5 / 45.1
constexpr int kTileMinAvg = 40, kTileMinAvgMany = 20, kTileMinAvgExact = 64, kTileManyItems = 768;
constexpr long long kTileMinOutputs = 7 << 18;

// Rows of stream_fp8's tiles, 16 * mf: 16 only where that leaves no CU a second item.  us with 16 / 32 rows: linear
// 2048 -> 2048, 256 rows (256 items of 16) 9.4 / 12.0, 300 rows 13.4 / 12.2; FFN of 8 groups of 16 rows, 1472 x 832,
// 18.7 / 21.3, of 128 groups of 8 rows, 2880 x 2880, 582 / 547, of 16 rows 637 / 559.
constexpr int kSmallItems = 256;

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
  const int tile_cols = m == kGateUp ? TileCodes::BN / 2 : TileCodes::BN;
  const bool many = static_cast<long long>(s.sequences()) * ((s.cols + tile_cols - 1) / tile_cols) >= kTileManyItems;
  const int least = exact ? kTileMinAvgExact : many ? kTileMinAvgMany : kTileMinAvg;
  if (avg >= least && area >= kTileMinOutputs && s.K > (kTileMinStages - 1) * kBlock && s.groups() <= kTileMostGroups)
    return Plan{exact ? Kernel::kTileExact : Kernel::kTile, 0, 0};
  const int nch = (s.cols + kBlock - 1) / kBlock, mf = static_cast<long long>(max_m_tiles(s, 16)) * nch <= kSmallItems ? 1 : 2;
  return Plan{Kernel::kStream, mf, item_grid(max_m_tiles(s, 16 * mf), nch)};
}

inline Plan linear_plan(bool exact, const Sizes& s) { return few_linear(s) ? few_plan(kLinear, s) : many_plan(kLinear, exact, s); }

// kGateUp: K = d, cols = I; kDown: K = I, cols = d.
inline Plan ffn_plan(Mode m, const Sizes& s) {
  return few_ffn(s.n_rows, m == kGateUp ? s.cols : s.K) ? few_plan(m, s) : many_plan(m, false, s);
}

}  // namespace fp8
}  // namespace moe
