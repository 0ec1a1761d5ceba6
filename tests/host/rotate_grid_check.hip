// Host-side check of the rotation's launches over every number of heads and token
// counts from 1 to the most of a launch: workgroups for every head of every token, and
// an extent of the grid below 2^32 threads.
#include <cstdio>

#include "rotary.h"

int main() {
  using namespace pmqa;
  long bad = 0, checked = 0;
  for (int heads = 1; heads <= IDX_MAX_ATTENTION_HEADS; ++heads) {
    for (int64_t power = 1; power <= IDX_MAX_APPEND_TOKENS; power *= 2) {
      for (int d = -3; d <= 3; ++d) {
        const int64_t all = power + d;
        if (all < 1 || all > IDX_MAX_APPEND_TOKENS) continue;
        const int32_t tokens = static_cast<int32_t>(all < kSlabTokens ? all : kSlabTokens);
        const uint64_t workgroups = rotate_workgroups(tokens, heads);
        const bool ok = workgroups * kRotateThreads < (uint64_t{1} << 32) &&
                        workgroups * kHeadsPerWg >= static_cast<uint64_t>(tokens) * heads &&
                        workgroups == static_cast<uint64_t>(tokens) * chunks_of(heads);
        if (!ok && bad++ < 10)
          std::printf("%d tokens of %d heads: %llu workgroups\n", tokens, heads, static_cast<unsigned long long>(workgroups));
        ++checked;
      }
    }
  }
  std::printf("checked %ld, mismatches %ld\n", checked, bad);
  return bad == 0 ? 0 : 1;
}
