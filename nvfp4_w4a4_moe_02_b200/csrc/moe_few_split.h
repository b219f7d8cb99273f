// How the few-token layer's streaming kernels split K: plain arithmetic, the same on the host.
#pragma once
#include "host_device.h"

namespace nvfp4 {

constexpr int kFewWarps = 16;  // warps of a block, and the most that split K

// The chunks of the busiest warp where teams of S = 2^i warps share the units evenly and split a unit's
// nch chunks, a join counted as one, with i in the low three bits.  The least over the 32 lanes i of a warp
// is the choice; a lane whose S is more than a block's warps or than the chunks never is,
// and does not divide: the warps shifted by its i may leave no team.
NVFP4_HOST_DEVICE uint32_t few_split_cost(int i, int units, int warps, int nch) {
  if ((kFewWarps >> i) == 0 || nch >> i == 0) return 0xFFFFFFFFu;
  const uint32_t teams = (uint32_t)warps >> i;
  const uint32_t busiest = ((uint32_t)units + teams - 1) / teams;
  return (busiest * (uint32_t)(((nch - 1) >> i) + 1 + (i > 0))) << 3 | (uint32_t)i;
}

}  // namespace nvfp4
