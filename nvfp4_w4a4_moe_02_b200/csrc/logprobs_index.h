// The backward pass's shares of a row: plain arithmetic, the same on the host.
#pragma once
#include "host_device.h"

namespace nvfp4 {

// Stretches of a row of V logits, N to a vector: four vectors a thread of 256, more where T rows of them
// would pass the grid's limit.
NVFP4_HOST_DEVICE int64_t logprob_stretches(int64_t T, int64_t V, int N) {
  const int64_t n = (V + 1024 * N - 1) / (1024 * N);
  return n < INT32_MAX / T ? n : INT32_MAX / T;
}

// The elements [first, end) of a stretch.  V goes to 2^31 - 1, and a counter that runs over them steps past
// the end by up to a team: unsigned, it neither overflows nor comes back below the end.
struct ElementRange {
  uint32_t first, end;
};
NVFP4_HOST_DEVICE ElementRange stretch_elements(int64_t V, int64_t at, int64_t stretches) {
  return {(uint32_t)(V * at / stretches), (uint32_t)(V * (at + 1) / stretches)};
}

}  // namespace nvfp4
