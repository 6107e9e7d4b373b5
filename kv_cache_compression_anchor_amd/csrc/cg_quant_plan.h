// How a call of the attention over caches held in 4 bits is launched, from its numbers alone:
// which kernel, and how the tokens are cut.  Plain C++: cg_quant_attention.hip launches by it,
// and so can a host program look it over.
#pragma once

#include <algorithm>

#include "cg_paged.h"
#include "cg_ranges.h"

namespace cg {

// How a workgroup holds rows: all of 16 or 32 in each wave, which share out heads and tokens; or
// 16 or 32 in each wave of one head, all of whose waves go through the same tiles.
enum { kFew16 = 0, kFew32 = 1, kMany16 = 2, kMany32 = 3, kModes = 4 };
constexpr bool is_many(int mode) { return mode >= kMany16; }
constexpr int tiles_of_rows(int mode) { return 1 + (mode & 1); }  // of 16, of a wave
constexpr int rows_in(int dp, int mode) {
  return 16 * tiles_of_rows(mode) * (is_many(mode) ? dp == 256 ? 4 : 8 : 1);
}
// Workgroups on a compute unit, as LDS and registers allow.
constexpr int resident4(int pre, int rest) {
  return tiles_of_rows(pre) == 2 || tiles_of_rows(rest) == 2 ? 1 : 2;
}

// How a launch cuts the sequences: splits, or parts, of what the join then adds up, or each sequence to one workgroup,
// which writes the outputs (a.direct).  Known to the compiler, each needs fewer registers (100 to 345 scalar
// values still wait in lanes of vector registers, and one of the 52 kernels, <128, kMany16, kFew16, kParts>,
// spills 4 vector registers) and half the code, which a workgroup of few tokens fetches for one use.
enum { kSplits = 0, kParts = 1, kAlone = 2, kCuts = 3 };

// The kernels there are: rows held alike, or those of a prefix as more rows than the rest's, which are few;
// waves of 32 rows of 256 channels would not fit their registers.
constexpr bool built(int dp, int pre, int rest, int cut) {
  if (dp == 256 && (tiles_of_rows(pre) == 2 || tiles_of_rows(rest) == 2)) return false;
  return pre == rest || (cut != kAlone && pre > rest && !is_many(rest));
}

constexpr int kMostListed = 4096;  // sequences whose tiles a workgroup adds up

// How many splits and row tiles the launch has, from the call's numbers alone.
struct Plan {
  int dp, pre_splits, rest_splits, pre_least, rest_least, pre_tiles, rest_tiles, pre_mode, rest_mode, pre_groups, pre_heads,
      rest_heads, turn, parts;
  bool direct;
  size_t words;
  int cut() const { return direct ? kAlone : parts ? kParts : kSplits; }
};

// The smallest that holds `rows`.  Waves of 32 rows of 256 channels would not fit their registers.
inline int mode_of(int64_t rows, int dp) {
  if (rows <= 16) return kFew16;
  if (dp == 256) return kMany16;
  return rows <= 32 ? kFew32 : rows <= 128 ? kMany16 : kMany32;
}

inline Plan plan_of(const cg_paged_cache& c, const cg_quant_form& f, const cg_attention& x) {
  Plan p;
  const int kv = f.channels / x.head_dim, G = x.n_heads / kv;
  p.dp = x.head_dim <= 64 ? 64 : x.head_dim <= 128 ? 128 : 256;
  // Row tiles with workgroups of their own: few enough that an item's number, over
  // all heads, sequences and splits, fits 31 bits.
  auto most = [&](int64_t items) { return std::max<int64_t>(1, (1 << 21) / std::max<int64_t>(1, items)); };
  const int64_t rows = (int64_t)std::max(1, std::min(x.max_q, x.n_q)) * G;
  p.rest_mode = mode_of(rows, p.dp);
  const bool shared = x.n_groups > 0 && x.max_prefix > 0;
  p.pre_groups = x.n_groups;
  // rows of an average group
  const int64_t pre_rows = std::max<int64_t>(1, x.n_groups ? (x.n_q + x.n_groups - 1) / x.n_groups : 1) * G;
  p.pre_mode = mode_of(pre_rows, p.dp);
  // Prefixes and the rest are one launch: two, one after the other, leave the chip half empty (64
  // requests on 9,216 shared and up to 600 own tokens: 40 + 38 us).  A group's rows are as many as a
  // sequence's or more (21 sequences of up to 5 rows on three prompts: 38 us, with 32 rows for
  // both 43); where not, or both are many, both are held as the one with more.
  if (!shared) p.pre_mode = p.rest_mode;
  if (p.pre_mode < p.rest_mode || (is_many(p.pre_mode) && is_many(p.rest_mode)))
    p.pre_mode = p.rest_mode = std::max(p.pre_mode, p.rest_mode);
  auto row_tiles = [&](int64_t items, int64_t rows, int mode) {
    return (int)std::min(most(items), (rows + rows_in(p.dp, mode) - 1) / rows_in(p.dp, mode));
  };
  p.rest_tiles = row_tiles((int64_t)x.n_seqs * kv, rows, p.rest_mode);
  p.pre_tiles = row_tiles((int64_t)x.n_groups * kv, pre_rows, p.pre_mode);
  const int64_t slots = 256 * resident4(p.pre_mode, p.rest_mode);
  const int64_t own = std::max(0, x.max_len - (shared ? x.max_prefix : 0));
  auto tiles_in = [](int64_t tokens) { return (tokens + kTile - 1) / kTile; };
  // kv heads of a workgroup, and tiles of a super tile: as many as waves are left for, and as LDS holds.
  const int waves = p.dp == 256 ? 4 : 8;
  const QuantRow row = quant_row(f);
  auto heads = [&](int n) {
    while (kv % n) n--;
    int cpr = 0;  // as the kernel has it, at most
    for (int head = 0; head < kv && head < 8 * n; head += n)
      cpr = std::max(cpr, n * row.head / 16 + ((row.scales + 2 * head * row.groups) % 16 + 2 * n * row.groups + 15) / 16);
    p.rest_heads = n;
    p.turn = waves / n;
    while ((p.turn * 512 * cpr + 1023) / 1024 * 1024 > 37 * 1024 / 2) p.turn--;
  };
  // Few tokens: one head a workgroup, whose waves share the tokens, in one kernel that writes the
  // outputs itself, without a join.  For 8 kv heads of 128 channels, that kernel and the other
  // way: one sequence of 768 tokens 16 and 20 us, of 1,536 tokens 22 and 20; 8 of 1,000 20 and 20,
  // of 1,536 24 and 21; 32 of 512 19 and 22, of 1,000 28 and 22; 64 of 256 20 and 22, of 512 29
  // and 22.  Sharing prefixes saves (sequences - 1) times their reading, not for little: 64
  // sequences with 128 tokens in common (9 MB) 17.6 and 18 to 19 us, 16 with 512 (9 MB) 17 and 17.
  constexpr int kSteps = 4;  // super tiles that a workgroup takes rather than have sums joined
  const int64_t saved = shared ? (int64_t)x.n_seqs * x.max_prefix * c.channels * 4 : 0;
  auto alone = [&] {
    p.pre_mode = p.rest_mode;
    p.pre_groups = 0;
    p.pre_splits = 0;
    p.pre_heads = 1;
    p.pre_least = p.rest_least = 1;
    p.rest_splits = 1;
    p.parts = 0;
    p.words = 4;
    return p;
  };
  heads(1);
  if (is_many(p.rest_mode)) p.turn = 1;
  const int64_t all = (int64_t)x.n_seqs * p.rest_tiles * kv, room = 256 * resident4(p.rest_mode, p.rest_mode);
  // More than 32 rows, whose join reads more: also long sequences whose workgroups fill the chip, and
  // those that fill half of it up to kHalf tiles.  For 8 kv heads of 128 channels with 4 query heads each,
  // this way and cut (us): 2, 3, 4 prompts of 512 queries on 9,216 tokens (128, 192, 256 workgroups on 256
  // slots) 358 and 239, 359 and 336, 358 and 391; 16 of 64 queries (128) on 512 tokens 33 and 44, on 1,024 52
  // and 73, on 81,920 3,086 and 1,690; 8 of 128 queries (128) on 2,048 90 and 93; one of 512 and one of a
  // single query (128, 56 of them without rows) on 81,920 3,080 and 1,585, and eight of a single one (576)
  // 5,459 and 6,110.  64 channels, 32 kv heads, 8 of 64 queries (256 on 512 slots) on 4,096 85 and 77.  32
  // of 5 drafts, 8 query heads each, on 1,000 to 9,216 tokens (256 on 512) 225 and 130.
  constexpr int kHalf = 64;
  p.direct = saved <= (int64_t)16 << 20 &&
             (is_many(p.rest_mode) ? all >= room || (all >= room / 2 && tiles_in(x.max_len) <= kHalf) ||
                                         tiles_in(x.max_len) <= kSteps
                                   : tiles_in(x.max_len) <= kSteps * p.turn && all * tiles_in(x.max_len) <= waves * room);
  if (p.direct) return alone();
  // Otherwise as many neighbours as there are waves, so that whole stretches of rows are read.
  if (!is_many(p.rest_mode)) heads(waves);
  p.pre_heads = is_many(p.pre_mode) ? 1 : p.rest_heads;
  // Tiles of a split, at least `least`: so many that the items are `slots` workgroups at
  // most, and at most kMostSplits splits, whose sums the join reads.  A workgroup's start and
  // end take as long as kWorth super tiles.  What is shorter than the call says is cut as often, down to kLeast
  // tiles, as all these workgroups run at once (64 sequences on 9,216 shared tokens, said to be up to
  // 147,456: 45 us, in splits as long as said 253).
  constexpr int kMostSplits = 256, kWorth = 8;
  auto cut = [&](int64_t items, int64_t tiles, int64_t slots, int least, int& splits, int& per) {
    const int64_t by = std::min<int64_t>(std::max<int64_t>(1, slots / items), kMostSplits);
    const int64_t n = std::max<int64_t>((tiles + by - 1) / by, least);
    splits = (int)std::max<int64_t>(1, (tiles + n - 1) / n);
    per = std::min(least, kLeast);
  };
  const int64_t columns = kv / p.rest_heads, items = std::max(1, x.n_seqs) * p.rest_tiles * columns;
  const int64_t pre_items = (int64_t)x.n_groups * (kv / p.pre_heads) * p.pre_tiles;
  // Prefixes and the rest get slots by their work; lengths are mostly below the greatest.  A tile
  // takes a workgroup of many rows a third of the time of one of few rows of all heads.
  const int64_t pre_work = !shared ? 0 : pre_items * tiles_in(x.max_prefix) / (is_many(p.pre_mode) && !is_many(p.rest_mode) ? 3 : 1);
  const int64_t work = items * tiles_in(own) / 2;
  const int64_t pre_slots = pre_work ? std::min(std::max(slots * pre_work / (pre_work + work), slots / 8), slots * 7 / 8) : 0;
  // whole splits of all sequences: the prefix, whose workgroups all take as long, gets what they leave (0
  // where there are more sequences than slots, each of which is one split then)
  const int64_t rest_slots = pre_slots ? std::min((slots - pre_slots + items / 2) / items * items, slots * 7 / 8) : slots;
  const int least = (int)std::min<int64_t>(kWorth, std::max<int64_t>(kLeast, items * tiles_in(own) / 256)) * (is_many(p.rest_mode) ? 2 : p.turn);
  cut(items, tiles_in(own), rest_slots, least, p.rest_splits, p.rest_least);
  p.parts = 0;
  // the sums of tiles fit 31 bits
  const bool listed = x.n_seqs <= kMostListed && (int64_t)x.n_seqs * c.max_blocks * c.page_tokens < (int64_t)1 << 35;
  // Lengths that differ: equal parts of all of them, where that is two or more for each row tile and
  // its heads, and a launch has all items (2^22 at most) at once.
  if (x.n_seqs > 1 && listed && work >= kWorth * p.turn * (slots - pre_slots) &&
      slots - pre_slots >= 2 * columns * p.rest_tiles && pre_items <= 1 << 21) {
    p.parts = (int)std::max<int64_t>(1, (slots - pre_slots) / (columns * p.rest_tiles));
    p.rest_least = kWorth / 2 * p.turn;
    p.rest_splits = (int)std::max<int64_t>(2, std::min<int64_t>(kMostSplits + 2, 2 + 4 * ((p.parts + x.n_seqs - 1) / x.n_seqs)));
  }
  p.pre_splits = 0;
  p.pre_least = kLeast;
  if (x.n_groups)  // the slots that the rest leaves
    cut(pre_items, shared ? tiles_in(x.max_prefix) : 0, p.parts ? pre_slots : std::max(slots / 8, slots - items * p.rest_splits),
        kLeast, p.pre_splits, p.pre_least);
  p.words = (size_t)(p.pre_splits + p.rest_splits) * x.n_q * x.n_heads * (x.head_dim + 2) + x.n_q + 4;
  return p;
}

}  // namespace cg
