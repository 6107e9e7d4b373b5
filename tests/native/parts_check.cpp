// The cutting of all sequences' tiles, laid end to end, into equal parts (csrc/cg_ranges.h), walked
// through as the kernels do: every tile is in one part, a sequence's parts are numbered from 0 and fewer than
// the launch has room for, and as many as the join is told.  And split_of() with other least lengths.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "cg_ranges.h"

using namespace cg;

static void need(bool ok, const char* what) {
  if (!ok) {
    std::printf("%s\n", what);
    std::exit(1);
  }
}

static void walk(const std::vector<int>& tiles, int parts, int splits, int least) {
  const int n = (int)tiles.size();
  std::vector<int> at(n + 1, 0), done(n, 0), seen(n, 0);
  int top = 0;
  for (int s = 0; s < n; s++) {
    at[s + 1] = at[s] + tiles[s];
    top = std::max(top, tiles[s]);
  }
  const int all = at[n], per = tiles_of_part(all, top, parts, splits, least);
  need(per >= least && per >= 1 && (int64_t)per * parts >= all, "tiles behind the last part");
  for (int part = 0; part < parts; part++) {
    int pos = (int)std::min((int64_t)part * per, (int64_t)all);
    const int end = std::min(pos + per, all);
    int s = (int)(std::upper_bound(at.begin(), at.end() - 1, pos) - at.begin()) - 1, base = at[s];
    while (pos < end && s < n) {
      const int q = s++;
      if (tiles[q] == 0) continue;
      const Parts in = parts_of(base, tiles[q], per);
      const int from = pos - base, m = std::min(tiles[q] - from, end - pos), split = part - in.first;
      need(from >= 0 && m > 0 && from == done[q], "a tile twice or never");
      need(split == seen[q] && split < in.used, "numbers of a sequence's parts");
      need(in.used <= splits, "more parts of a sequence than there is room for");
      done[q] += m;
      seen[q]++;
      if (done[q] == tiles[q]) need(seen[q] == in.used, "the join is told another number of parts");
      pos += m;
      base += tiles[q];
    }
    need(pos == end, "a part that ends early");
  }
  need(done == tiles, "tiles lost");
}

int main() {
  std::mt19937 rng(3);
  auto upto = [&](int64_t n) { return (int)(rng() % (uint64_t)(n + 1)); };
  for (int tries = 0; tries < 6000; tries++) {
    const int n = 1 + (upto(3) ? upto(40) : upto(4095)), most = 1 << upto(11);
    std::vector<int> tiles(n);
    for (int& t : tiles) t = upto(3) ? upto(most) : 0;
    walk(tiles, 1 + upto(511), 2 + upto(256), 1 + upto(64));
  }
  // the longest rows (2^30 tokens), as many as the sums of tiles allow
  const int longest = (1 << 30) / kTile;
  for (int n : {1, 2, 31, 32})
    for (int parts : {1, 2, 3, 511, 512})
      for (int splits : {2, 3, 258})
        for (int least : {1, 4, 32}) {
          std::vector<int> tiles(n, longest);
          walk(tiles, parts, splits, least);
          if (n > 2) tiles[1] = 0, tiles[n - 1] = 1;
          walk(tiles, parts, splits, least);
        }
  const int lens[] = {0, 1, 31, 32, 33, 127, 128, 129, 1000, 100000, (1 << 30) - 1, 1 << 30};
  for (int lo : lens)
    for (int hi : lens)
      for (int splits : {0, 1, 2, 3, 7, 64, 256})
        for (int least : {1, 2, 4, 7, 56, 64}) {
          const Split s = split_of(lo, hi, splits, least);
          need(s.per >= least && s.tiles >= 0 && s.used >= 0 && s.used <= std::max(1, splits), "split_of");
          need((int64_t)s.used * s.per >= s.tiles && (s.used == 0 || (int64_t)(s.used - 1) * s.per < s.tiles), "tiles lost");
        }
  std::printf("parts ok\n");
}
