// Reads lines "T V N at" (at = -1: every stretch, -2: the last one) and checks that the threads of a stretch
// take each of its elements once and nothing else.  Built with the undefined-behaviour checks on.
#include <cstdio>
#include <vector>

#include "logprobs_index.h"

int main() {
  long long T, V, N, at;
  while (std::scanf("%lld %lld %lld %lld", &T, &V, &N, &at) == 4) {
    const int64_t n = nvfp4::logprob_stretches(T, V, (int)N);
    if (n < 1 || n * T > INT32_MAX) return std::printf("grid of %lld x %lld\n", T, (long long)n), 1;
    int64_t next = at == -2 ? V * (n - 1) / n : 0;
    for (int64_t s = at == -2 ? n - 1 : 0; s < n; ++s) {
      const int64_t lo = next;
      std::vector<int> seen((size_t)(V * (s + 1) / n - lo), 0);
      const nvfp4::ElementRange r = nvfp4::stretch_elements(V, s, n);
      for (int tid = 0; tid < 256; ++tid)
        for (auto v = r.first + tid; v < r.end; v += 256) {  // as the kernel's loop
          if (v < lo || v - lo >= (int64_t)seen.size()) return std::printf("element %lld of %lld\n", (long long)v, V), 1;
          ++seen[(size_t)(v - lo)];
        }
      for (int c : seen)
        if (c != 1) return std::printf("an element taken %d times\n", c), 1;
      next = lo + (int64_t)seen.size();
    }
    if (next != V) return std::printf("the last stretch ends at %lld of %lld\n", (long long)next, V), 1;
  }
  std::printf("ok\n");
}
