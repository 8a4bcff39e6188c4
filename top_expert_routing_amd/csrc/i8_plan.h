// Which kernel runs an int8 product (ffn_i8.hip) and how much LDS its tiles take, from the
// sizes alone: host arithmetic without GPU code, so that a host program can ask it too.
#pragma once

#include "item_plan.h"

namespace moe {
namespace i8 {

enum Mode { kLinear, kGateUp, kDown };   // products: described at the kernels

constexpr int kLanes = 64;           // of a wavefront
constexpr int kBlock = 128;          // columns of the SwiGLU product that share a scale
constexpr int kStep = 64;            // K of one matrix instruction

// ---- tile_i8's tiles and their LDS ---------------------------------------------------
template <int MI_, int NJ_, int WM_, int WN_, int BPC_>
struct TileCfg {
  static constexpr int BPC = BPC_;                             // blocks per CU
  static constexpr int MI = MI_, NJ = NJ_, WM = WM_, WN = WN_, NW = WM * WN, NT = kLanes * NW;
  static constexpr int BM = 16 * MI * WM, BN = 16 * NJ * WN;
  static constexpr int ADMA = BM / 16 / NW, BDMA = BN / 16 / NW;
  static_assert(ADMA >= 1 && ADMA <= 4 && BDMA >= 1, "DMA instructions per wave");
};
constexpr int kLdsPerCu = 160 * 1024;
constexpr int kTileMinK = 4 * kStep;   // shortest K of tile_i8 (TileLds)
template <class C, Mode M>
struct TileLds {
  static constexpr int SUB = M == kDown ? 2 : 1;               // K steps per stage
  static constexpr int A = C::BM * kStep, B = C::BN * kStep;   // bytes per K step
  static constexpr int WROWS = 16 * C::ADMA * 4;               // one 4-byte value per row: of a wave's loads, of all
  static constexpr int ROWS = C::NW * WROWS;
  static constexpr int STAGE = SUB * (A + B) + (M == kDown ? ROWS : 0);
  // as many as fit beside 12 KiB (two blocks per CU: 8) of lists, scales and the plan
  static constexpr int STAGES = (kLdsPerCu / C::BPC - (C::BPC == 2 ? 8 : 12) * 1024) / STAGE;
  static constexpr int AHEAD = STAGES - 1;                     // stages requested before the first is used
  static_assert(STAGES >= 2 && (M != kGateUp || C::BN == 2 * kBlock), "a kGateUp tile holds the columns of one scale");
  // The stages requested before a block's first product stop short of its first tile's last one: what
  // follows it is the next tile's, whose sources are set when the first tile starts.
  static_assert(kTileMinK / (kStep * SUB) > AHEAD, "a tile has more stages than are requested ahead");
  static constexpr int RING = STAGES * STAGE;
  static constexpr int LIST = RING;                            // row list of two tiles
  static constexpr int SA = LIST + 2 * ROWS;                   // row scales of two tiles
  static constexpr int SB = SA + 2 * ROWS;                     // channel scales of two tiles
  static constexpr int MAX = SB + 2 * 1024;                    // kGateUp: largest magnitudes
  static constexpr int PLAN = MAX + C::WN * C::BM * 4;         // sums over waves, tiles before each group, group offsets
  static int bytes(int G) { return PLAN + 4 * C::NW + 8 * (G + 1); }
};

using TileWide = TileCfg<4, 8, 4, 2, 1>;   // 256 rows, one block of eight waves per CU
using TileHalf = TileCfg<4, 8, 2, 2, 2>;   // 128 rows, two blocks of four waves per CU

// ---- which kernel ----------------------------------------------------------------------
// The host sees the average group, not the groups; items are counted against the MI355X's 256
// CUs.  Times of the whole call,
// us; d, I or K, O = 2048, 1024 (FFN, 64 groups) and 2048, 2048 (linear, one group).
//   few_i8 or stream_i8     linear 16 rows 4.8 / 6.7, 128 rows 6.1 / 6.8, 256 rows 9.9 /
//                           7.2: few_i8 up to kFewBlocksMost items of 16 x 16 (1024 x 512,
//                           512 rows 5.5 / 5.6, 1024 rows 9.2 / 7.1).  FFN with 8 groups of
//                           one row 16.2 / 18.4, of 8 rows 23.8 / 19.2; 16 groups of one
//                           row, 1024 x 512, 11.8 / 13.4; 64 groups of one row 106 / 75:
//                           only up to kFewItems items of 128 columns, which also bounds the
//                           fp32 product to 80 KiB.
//   stream_i8 or tile_i8    64 rows a group 108 / 109, 96 rows 137 / 117; but linear 2048
//                           rows (512 items of 64 x 128) 23 / 26, 5800 rows x 2112 -> 832
//                           (589) 35 / 30, 4096 rows (1024) 43 / 31, 16 groups of 256
//                           rows, 1024 x 512 (256 items) 33 / 39: tile_i8 needs both full
//                           tiles and enough of them.  By the product of an FFN: gate/up
//                           384 items 85 / 92, 528 items 93 / 87, 611 items 69 / 58; down 500
//                           items 57 / 66, 700 items 69 / 76, 917 items 82 / 69.
//   TileHalf or TileWide    128 rows a group 125 / 130, 192 rows 156 / 147; linear 4096 rows
//                           (128 wide tiles) 32 / 34, 8191 x 4096 (512) 75 / 70.
// Averages are rows per sequence that tiles are cut from (Sizes::sequences), not per group: with
// 64 priority tokens, 128 experts x 4, 2880 x 2880, by group / by sequence: 1024 tokens 985 / 746,
// 2560 tokens 1229 / 831, 4096 tokens 1535 / 967, 4160 tokens 969 / 966, 6144 tokens 1214 / 1084;
// 64 experts x 8, 2048 x 1024: 256 tokens 136 / 109, 1024 tokens 211 / 152, 2048 tokens 212 / 181.
constexpr int kFewItems = 160, kFewBlocks = 384, kFewBlocksMost = 1024;
constexpr int kIdleLinear = 200, kIdleFfn = 256;
constexpr int kTileMinAvg = 64;
constexpr int tile_min_items(Mode m) { return m == kGateUp ? 512 : m == kDown ? 736 : 576; }
constexpr int kWideMinAvg = 192, kWideMinTiles = 256;

// Rows of stream_i8's tiles, 16 * mf: 16 for groups that mostly fit (64 groups, 2048 x 1024, with
// 16 and 32 rows a tile: of 12 rows 79 / 81 us, of 24 rows 88 / 86).  No more than 32: items
// of the same weights then read them from the L2, but more of them fit on a CU (64 rows a tile: FFN of
// 481 tokens x 8 of 128 experts, 2240 x 640, 202 us against 161; 700 x 4 of 8, 1472 x 832, 51
// against 43; a single group of 2048 rows x 2048 -> 2048 21 against 23).  Where CUs are left without
// an item (at most kIdle... of them), 16 rows: us without / with: linear 300 rows x 2048 -> 1024
// 8.4 / 6.8; FFN of 8 groups of 32 rows, 2048 x 1024, 22.6 / 20.3.  At 200 or 256 items: linear 512
// rows 8.8 / 10.0, FFN 16 groups of 64 rows, 1024 x 512, 18.6 / 17.3.
inline int pick_mf(int avg) { return avg <= 16 ? 1 : 2; }

// A product of n_rows sorted rows in nseg * E + n_shared groups with matrices [cols][K].
struct Sizes {
  int n_rows, E, n_shared, nseg, K, cols;
  int groups() const { return nseg * E + n_shared; }
  // Row sequences that tiles are cut from: an expert's rows of both segments form one (group_rows).
  int sequences() const { return E + n_shared; }
};

// The FFN's products of few rows (both of them: the SwiGLU product is kept in fp32 then).
inline bool few(int n_rows, int I) { return static_cast<long long>(n_rows) * ((I + kBlock - 1) / kBlock) <= kFewItems; }

// m-tiles of BM rows of a call, at most: ceil(n / BM) <= 1 + (n - 1) / BM for each sequence with rows.
inline int max_m_tiles(const Sizes& s, int BM) {
  const int sequences = s.sequences() < s.n_rows ? s.sequences() : s.n_rows;
  return sequences + (s.n_rows - sequences) / BM;
}

enum class Kernel { kFew, kStream, kTileHalf, kTileWide };
struct Plan {
  Kernel kernel;
  int width;    // few_i8: 16-column blocks of an item; stream_i8: 16-row blocks of a tile
  int blocks;   // few_i8, stream_i8: blocks of the launch (tile_i8's walk a list)
};

// The launch of a plan's blocks: those past 2^20 lie along y, because a grid has fewer than 2^32
// threads along x (2^20 is a multiple of the XCDs, so block y * kMostX + x goes to XCD x % 8 as ever).
constexpr int kMostX = 1 << 20;
struct Launch {
  int x, y;
};
inline Launch launch_of(const Plan& p) {
  return p.blocks <= kMostX ? Launch{p.blocks, 1} : Launch{kMostX, (p.blocks - 1) / kMostX + 1};
}

inline Plan plan_few(Mode m, const Sizes& s) {
  const int tiles = max_m_tiles(s, 16), blocks16 = tiles * (s.cols / 16);
  // wider items where 16 columns give more blocks than run at once (a block is mostly waits:
  // 1024 of them took 10.7 us for one token's down product, 256 of 64 columns 5 us)
  const int nc = blocks16 <= kFewBlocks ? 1 : m == kGateUp || blocks16 <= 2 * kFewBlocks ? 2 : 4;
  return Plan{Kernel::kFew, nc, item_grid(tiles, s.cols / (16 * nc))};
}

inline Plan plan_many(Mode m, const Sizes& s) {
  const int avg = s.n_rows / s.sequences();
  const long long area = static_cast<long long>(s.n_rows) * s.cols;
  if (avg > kTileMinAvg && s.K >= kTileMinK && area >= tile_min_items(m) * 64ll * 128) {
    const long long wide = area / (256 * (m == kGateUp ? 128 : 256));
    // (the lists of two blocks per CU have room for some 380 groups)
    const int half_lds = m == kGateUp ? TileLds<TileHalf, kGateUp>::bytes(s.groups()) : TileLds<TileHalf, kLinear>::bytes(s.groups());
    const bool big = m == kDown || (avg >= kWideMinAvg && wide >= kWideMinTiles) || half_lds > kLdsPerCu / 2;
    return Plan{big ? Kernel::kTileWide : Kernel::kTileHalf, 0, 0};
  }
  const int nch = (s.cols + kBlock - 1) / kBlock;
  int mf = pick_mf(avg);
  if (max_m_tiles(s, 16 * mf) * nch <= (m == kLinear ? kIdleLinear : kIdleFfn)) mf = 1;
  return Plan{Kernel::kStream, mf, item_grid(max_m_tiles(s, 16 * mf), nch)};
}

inline Plan plan_linear(const Sizes& s) {
  return static_cast<long long>(max_m_tiles(s, 16)) * (s.cols / 16) <= kFewBlocksMost ? plan_few(kLinear, s)
                                                                                      : plan_many(kLinear, s);
}

// kGateUp: K = d, cols = I; kDown: K = I, cols = d.
inline Plan plan_ffn(Mode m, const Sizes& s) {
  return few(s.n_rows, m == kGateUp ? s.cols : s.K) ? plan_few(m, s) : plan_many(m, s);
}

}  // namespace i8
}  // namespace moe
