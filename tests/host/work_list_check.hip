// Host-side check of the choice of the attention's pair tiles: whatever the estimated
// times of the sizes, the work list of the chosen size fits the counters in which the
// kernel adds it up.  Rows, heads and requests from one to the most, uniform and
// ragged, and tables of times that make each size the best wherever it may be taken.
#include <cstdio>

#include "attention_common.h"

namespace {
using namespace pmqa;
long bad = 0, checked = 0;

template <int KIND>
void check(const AttentionArgs& a) {
  constexpr double kFixed[4] = {};
  for (int best = 0; best < 4; ++best) {
    double per_tile[4] = {1e9, 1e9, 1e9, 1e9};
    per_tile[best] = 1e-9;
    for (const int64_t narrowest : {ScanOf256<KIND>::kItems, ScanOf512<KIND>::kItems}) {
      const int m = tile_pairs<KIND>(a, per_tile, kFixed, narrowest);
      const int64_t items = item_count<KIND>(a, m), most = m == 16 ? narrowest : ScanOf256<KIND>::kItems;
      if (items > most && bad++ < 10)
        std::printf("kind %d rows %d heads %d requests %d ragged %d: %d pairs, %lld items\n", KIND, a.rows, a.heads,
                    a.requests, a.cu_q != nullptr, m, static_cast<long long>(items));
      ++checked;
    }
  }
}
}  // namespace

int main() {
  int32_t cu_q = 0;
  for (int heads = 1; heads <= IDX_MAX_ATTENTION_HEADS; ++heads) {
    for (int requests : {1, 2, 3, 64, 100, 1000, 1285, 4095, 4096}) {
      for (int next_n : {0, 1, 2, 4, 15, 16, 51, 100, 1000, 21845, 32767, 65535}) {
        for (int rows : {requests, 1 << 10, 20000, 32768, IDX_MAX_ROWS}) {
          if (next_n) rows = requests * next_n;
          if (rows > IDX_MAX_ROWS) continue;
          AttentionArgs a{};
          a.rows = rows;
          a.heads = heads;
          a.requests = requests;
          a.next_n = next_n;
          a.cu_q = next_n ? nullptr : &cu_q;
          a.k = 2048;
          a.max_pages = 512;
          a.prefix_pages = 1;
          check<kDense>(a);
          check<kSparse>(a);
          if (next_n) check<kShared>(a);
        }
      }
    }
  }
  std::printf("checked %ld, mismatches %ld\n", checked, bad);
  return bad == 0 ? 0 : 1;
}
