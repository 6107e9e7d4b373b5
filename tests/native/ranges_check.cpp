// The attention's ranges of queries and tokens (csrc/cg_ranges.h) on numbers from both
// ends of the type, against 64-bit arithmetic, and as the kernels' loops use them.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "cg_ranges.h"

using namespace cg;

static void need(bool ok, const char* what) {
  if (!ok) {
    std::printf("%s\n", what);
    std::exit(1);
  }
}

int main() {
  const int32_t ends[] = {INT32_MIN, INT32_MIN + 1, -1, 0, 1, 2, 5, 6, 7, 255, 256, 1 << 20, INT32_MAX - 1, INT32_MAX};
  for (int n_q : {0, 1, 6, 1 << 20})
    for (int32_t start : ends)
      for (int32_t end : ends) {
        const int64_t m = (int64_t)end - start;
        need(queries_of(start, end, n_q) == (start >= 0 && end <= n_q && m > 0 ? m : 0), "queries_of");
        // a workgroup's threads over the queries
        for (int thread : {0, 1, 63, 255})
          for (int i = begin_of(start, n_q) + thread; i < end_of(end, n_q); i += 256)
            need(i >= 0 && i < n_q && i >= start && i < end, "a query outside the batch");
      }
  const int32_t lens[] = {0, 1, 31, 32, 33, 127, 128, 129, 1000, 100000, (1 << 30) - 1, 1 << 30};
  for (int32_t lo : lens)
    for (int32_t hi : lens)
      for (int splits : {0, 1, 2, 3, 7, 64}) {
        const Split s = split_of(lo, hi, splits);
        need(s.per >= kLeast && s.tiles >= 0 && s.used >= 0, "split_of");
        need(s.used <= (splits < 1 ? 1 : splits), "more splits than there are");
        need((int64_t)s.used * s.per >= s.tiles && (s.used == 0 || (int64_t)(s.used - 1) * s.per < s.tiles), "tiles lost");
        need(hi <= lo ? s.tiles == 0 && s.used == 0
                      : (int64_t)s.tile0 * kTile <= lo && (int64_t)(s.tile0 + s.tiles) * kTile >= hi,
             "tokens lost");
      }
  std::printf("ranges ok\n");
}
