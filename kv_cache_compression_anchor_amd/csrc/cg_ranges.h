// Ranges of queries and tokens, worked out from numbers in device memory that may be
// anything.  Plain C++: the attention's kernels use these, and so can a host program.
#pragma once

namespace cg {

constexpr int kTile = 32;  // tokens of a tile: the depth of one 16x16x32 product
// Tiles of a split, at least: one for each wave.  With more, short contexts leave most
// of the chip idle (8 requests of 20 heads, 5 of K and V, on 992 shared and 630 own tokens:
// 17 us with 4, 18 with 8, 24 with 16).
constexpr int kLeast = 4;

// Queries start .. end - 1 of a batch of n_q: how many, none where the starts descend
// or leave the batch (their difference may wrap around).
constexpr int queries_of(int start, int end, int n_q) {
  return start >= 0 && end > start && end <= n_q ? end - start : 0;
}
// The same as far as the batch has them: from begin_of to end_of.
constexpr int begin_of(int start, int n_q) { return start < 0 ? 0 : start < n_q ? start : n_q; }
constexpr int end_of(int end, int n_q) { return end < n_q ? end : n_q; }

// Tokens [lo, hi) in tiles that start at multiples of kTile, dealt to `splits`
// workgroups in turn, at least kLeast each.  Without tokens there may be no splits.
struct Split {
  int tile0, tiles, per, used;
};
constexpr Split split_of(int lo, int hi, int splits) {
  Split s{lo / kTile, hi > lo ? (hi + kTile - 1) / kTile - lo / kTile : 0, 0, 0};
  if (splits < 1) splits = 1;
  s.per = (s.tiles + splits - 1) / splits;
  if (s.per < kLeast) s.per = kLeast;
  s.used = (s.tiles + s.per - 1) / s.per;
  return s;
}

}  // namespace cg
