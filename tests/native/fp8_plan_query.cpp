// Prints the kernel that the library picks for FP8 products: one line
// "product n_rows E n_shared nseg K cols" in (product: linear, linear_f32, gate_up, down), one line
// "kernel width blocks x y" out (x, y: the launch's grid).
#include <cstdio>
#include <cstring>

#include "../../top_expert_routing_amd/csrc/fp8_plan.h"

using namespace moe::fp8;

// every layout that the kernels use: its static_asserts hold
template struct moe::fp8::TileLds<TileCodes, kLinear>;
template struct moe::fp8::TileLds<TileCodes, kGateUp>;
template struct moe::fp8::TileLds<TileCodes, kDown>;
template struct moe::fp8::TileLds<TileExact, kLinear>;

int main() {
  char product[16];
  Sizes s;
  while (std::scanf("%15s %d %d %d %d %d %d", product, &s.n_rows, &s.E, &s.n_shared, &s.nseg, &s.K, &s.cols) == 7) {
    const Plan p = std::strncmp(product, "linear", 6) ? ffn_plan(std::strcmp(product, "down") ? kGateUp : kDown, s)
                                                      : linear_plan(!std::strcmp(product, "linear_f32"), s);
    const char* names[] = {"few", "stream", "tile_codes", "tile_exact"};
    const Launch l = launch_of(p);
    std::printf("%s %d %d %d %d\n", names[static_cast<int>(p.kernel)], p.width, p.blocks, l.x, l.y);
  }
  return 0;
}
