// Host-side check of the rotation's grid over every number of heads and token counts
// from 1 to the most: an extent in threads stays below 2^32, every token has its
// workgroups in one slab, and no slab is empty.
#include <cstdio>

#include "rotary.h"

int main() {
  using namespace pmqa;
  long bad = 0, checked = 0;
  for (int heads = 1; heads <= IDX_MAX_ATTENTION_HEADS; ++heads) {
    for (int32_t power = 1; power <= IDX_MAX_APPEND_TOKENS; power *= 2) {
      for (int d = -3; d <= 3; ++d) {
        const int32_t tokens = power + d;
        if (tokens < 1 || tokens > IDX_MAX_APPEND_TOKENS) continue;
        const RotateGrid g = rotate_grid(tokens, heads);
        const uint64_t threads = static_cast<uint64_t>(g.x) * kRotateThreads;
        const uint64_t side = g.x / g.chunks;  // tokens of a slab
        const bool ok = threads < (uint64_t{1} << 32) && g.z >= 1 && g.z <= 65535 && g.x % g.chunks == 0 &&
                        g.chunks * kHeadsPerWg >= heads && (g.z == 1 || side == kSlabTokens) &&
                        g.z * side >= static_cast<uint64_t>(tokens) && (g.z - 1) * side < static_cast<uint64_t>(tokens);
        if (!ok && bad++ < 10) std::printf("%d tokens of %d heads: grid %u x %u\n", tokens, heads, g.x, g.z);
        ++checked;
      }
    }
  }
  std::printf("checked %ld, mismatches %ld\n", checked, bad);
  return bad == 0 ? 0 : 1;
}
