// Prints the kernel that the library picks for int8 products: one line
// "product n_rows E n_shared nseg K cols" in (product: linear, gate_up, down), one line
// "kernel width blocks x y" out (x, y: the launch's grid).
#include <cstdio>
#include <cstring>

#include "../../top_expert_routing_amd/csrc/i8_plan.h"

using namespace moe::i8;

// every layout that the kernels use: its static_asserts hold
template struct moe::i8::TileLds<TileWide, kLinear>;
template struct moe::i8::TileLds<TileWide, kGateUp>;
template struct moe::i8::TileLds<TileWide, kDown>;
template struct moe::i8::TileLds<TileHalf, kLinear>;
template struct moe::i8::TileLds<TileHalf, kGateUp>;

int main() {
  char product[16];
  Sizes s;
  while (std::scanf("%15s %d %d %d %d %d %d", product, &s.n_rows, &s.E, &s.n_shared, &s.nseg, &s.K, &s.cols) == 7) {
    const Plan p = !std::strcmp(product, "linear") ? plan_linear(s)
                                                   : plan_ffn(std::strcmp(product, "down") ? kGateUp : kDown, s);
    const char* names[] = {"few", "stream", "tile_half", "tile_wide"};
    const Launch l = launch_of(p);
    std::printf("%s %d %d %d %d\n", names[static_cast<int>(p.kernel)], p.width, p.blocks, l.x, l.y);
  }
  return 0;
}
