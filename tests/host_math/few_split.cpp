// Reads lines "units warps nch" and prints the team size S that the 32 lanes of a warp choose.  Built with
// the undefined-behaviour checks on: a division by zero in any lane ends the program.
#include <algorithm>
#include <cstdio>

#include "moe_few_split.h"

int main() {
  int units, warps, nch;
  while (std::scanf("%d %d %d", &units, &warps, &nch) == 3) {
    uint32_t least = 0xFFFFFFFFu;
    for (int lane = 0; lane < 32; ++lane) least = std::min(least, nvfp4::few_split_cost(lane, units, warps, nch));
    std::printf("%d\n", 1 << (least & 7u));
  }
}
