// Attention over a paged cache held in 4 bits (include/cachegen.h, cg_quant_attention_async).
//
// The method is cg_attention.hip's: any split of the tokens, sums against reference
// exponents that join.  The numbers s n of the cache are binary16 numbers, and are made in
// registers on the way to the products:
//   nibbles n + 8 of a 32-bit word, two at a time, become halves 1024 + (n + 8) or
//   64 + (n + 8) by one and-or (they are the low mantissa bits of 1024, or of 64), a
//   subtraction leaves n exactly, a product with s is exact by the form of s.
// The products and the softmax are cg_attention.h's: S^T = K Q^T and O^T = V^T P^T by 16 x 16 x 32
// products of binary16 into binary32, sums and references in binary32, the weights rounded to
// binary16 (what the second product takes; 2^-11 of a weight at most).
//
// One launch for shared prefixes and the sequences' own tokens, and k_join where tokens were cut.  Few
// rows (up to 32 of a kv head): a workgroup of eight waves takes eight kv heads of a tile, whole
// stretches of rows come to LDS, and each wave makes its head's numbers in registers.  More rows:
// all waves take one head, whose numbers are made once, into LDS.
//
// What bounds it: 64 sequences of 1,000 to 9,216 tokens (32 heads, 8 of K and V, 128 channels, 345 MB)
// take 93 us with the join, which takes 7 (70.7 at a copy's rate): vector instructions fill 75% of
// the issue slots, 3.35 a lane for a number of the cache, 1.7 of them to make it.  Four of 81,920
// tokens (378 MB) take 92 us.  64 on 9,216 shared tokens and up to 600 of their own take 44 with the join (7), at
// 1.3 us a tile of a workgroup (products and the numbers' making share the issue slots, two waves to
// each, and all waves do the same at one time) and 8 us of beginning and end.  Four prompts of 512 queries on
// 9,216 tokens take 360 us, 233 at the rate of a large product.
#include <algorithm>

#include "cg_attention.h"
#include "cg_hostapi.h"
#include "cg_quant_plan.h"

namespace cg {
namespace {

struct QuantAttn : Attn {
  int head_bytes, groups, scales;  // of a head: codes, scales; where the scales begin
  uint32_t row_bytes, page_bytes;
  int pre_least, rest_least;  // tiles of a split, at least
  int turn;                   // tiles of a super tile
  int pre_heads;              // kv heads of a workgroup of a shared prefix
  bool direct;                // one item has all of its queries' tokens and writes the outputs
  // not 0: the tiles of all sequences' own tokens, one sequence's behind the other's, are cut
  // into so many equal parts for each (row tile, kv heads), a workgroup each
  int parts;
};
__device__ __forceinline__ int prefix_heads(const QuantAttn& a) { return a.pre_heads; }

// Tiles [from, to) of a stretch of tokens.
struct Span {
  int from, to;
};
__device__ __forceinline__ Span span_of(int lo, int hi, int split, int splits, int least) {
  const Split s = split_of(lo, hi, splits, least);
  const int from = s.tile0 + split * s.per;
  return split < s.used ? Span{from, min(from + s.per, s.tile0 + s.tiles)} : Span{0, 0};
}

// ---------------------------------------------------------------------------
// Numbers
// ---------------------------------------------------------------------------
// The masks and exponents of the nibbles as values that the compiler does not know, masks in
// scalar and exponents in vector registers: an and-or takes no literals, and with known
// values becomes an and and an or.
struct Nibbles {
  uint32_t mask0 = 0x000F000Fu, mask1 = 0x00F000F0u, exp0 = 0x64006400u, exp1 = 0x54005400u;
  __device__ __forceinline__ Nibbles() { asm volatile("" : "+s"(mask0), "+s"(mask1), "+v"(exp0), "+v"(exp1)); }
  // Nibbles 0 and 4 (kHigh: 1 and 5) of a word, less 8, as halves.
  template <bool kHigh>
  __device__ __forceinline__ h2 get(uint32_t w) const {
    const uint32_t x = kHigh ? (w & mask1) | exp1 : (w & mask0) | exp0;
    const _Float16 bias = kHigh ? -72.0f : -1032.0f;
    return __builtin_bit_cast(h2, x) + h2{bias, bias};
  }
  // 8 channels of a word, in order, times s.
  __device__ __forceinline__ h8 numbers(uint32_t w, h2 s) const {
    const h2 a = get<false>(w) * s, b = get<true>(w) * s, c = get<false>(w >> 8) * s, d = get<true>(w >> 8) * s;
    return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
};
__device__ __forceinline__ h2 both(uint16_t s) {
  const _Float16 x = __builtin_bit_cast(_Float16, s);
  return h2{x, x};
}

// ---------------------------------------------------------------------------
// Super tiles of codes and scales in LDS
// ---------------------------------------------------------------------------
// A workgroup takes `heads` neighbouring kv heads of its tokens: of each token's row of K and
// of V one stretch of codes and one of scales.  A super tile is `turn` tiles of 32 tokens,
// brought to LDS as whole stretches by all waves; each wave then computes one head of one of its tiles.
// (Waves that bring their own heads' parts, 64 and 8 bytes of a row at a time, reach 4.0 TB/s
// with nothing else to do, 5.3 without the scales: half of what moves between the caches is
// not asked for.)
//   In LDS a row is `cpr` 16-byte chunks: the codes, then the scales' stretch from a multiple of
//   16 bytes on.  A head's chunk c (of DP / 32) of row r of a half tile lies at c ^ twist(r), which
//   spreads 16 rows of one chunk over the banks.
template <int DP>
struct Geo4 {
  static constexpr int kWaves = DP == 256 ? 4 : 8, kThreads = 64 * kWaves;
  static constexpr int CH = DP / 32;                  // chunks of a head of DP channels
  static constexpr int kStage = 37 * 1024;            // bytes of a super tile, two of which are in LDS
  static constexpr int kBlocks = (kStage / 2048 + kWaves - 1) / kWaves;  // loads of a wave of K, at most, and of V
  __device__ __forceinline__ static int twist(int r) { return CH == 2 ? (r >> 3) & 1 : CH == 4 ? (r >> 2) & 3 : (r >> 1) & 7; }
};

// LDS <- global, 16 bytes a lane, lane i's at lds + 16 i.  The compiler does not count these
// loads (wait_loads does), and a load takes m0 one wait state after its write.
__device__ __forceinline__ void load_lds(uint32_t lds, const char* addr) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(lds), "v"(addr) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// This thread's number, as a value that the compiler does not know: what is computed from it
// outside the loop over tiles is not kept in registers through it.
__device__ __forceinline__ int rare_thread() {
  int x = threadIdx.x;
  asm volatile("" : "+v"(x));
  return x;
}

// The pages of a stretch of tokens [lo, hi) of a table row, staged in LDS.
struct Pages {
  const int32_t* list;  // pages of blocks block0 .., -1 outside the pool
  int block0, lo, hi, shift, pmask;
  // Where token t's row is in a pool; of a token that does not exist some row.
  __device__ __forceinline__ uint64_t row_at(int t, uint32_t page_bytes, uint32_t row_bytes) const {
    const int page = max(list[(min(max(t, lo), hi - 1) >> shift) - block0], 0);
    return (uint64_t)(uint32_t)page * page_bytes + (uint64_t)(uint32_t)(t & pmask) * row_bytes;
  }
};

// Bits of the tokens of tile t0 that exist.
__device__ __forceinline__ uint32_t find(const Pages& p, int t0) {
  const int t = t0 + (rare_lane() & 31), c = min(max(t, p.lo), p.hi - 1);
  return (uint32_t)__ballot(t == c && p.list[(c >> p.shift) - p.block0] >= 0);
}

// What a workgroup's super tiles are like.
struct Columns {
  int heads, first;      // kv heads, the first of them
  int cpr, codes;        // chunks of a row in LDS, those of codes
  int window, skew;      // where the scales' stretch begins in a row of the cache, and the first head's in it
  int turn, vat;         // tiles; where V begins in a stage
  template <class A>
  __device__ __forceinline__ Columns(const A& a, int head, int n) : heads(n), first(head) {
    codes = n * a.head_bytes / 16;
    const int at = a.scales + 2 * head * a.groups;
    window = at & ~15;
    skew = at & 15;
    cpr = codes + (skew + 2 * n * a.groups + 15) / 16;
    turn = a.turn;
    vat = (turn * 512 * cpr + 1023) & ~1023;
  }
};

// A wave's part in bringing super tiles: blocks of 64 chunks, wave, wave + kWaves, .. of K's
// and the same of V's.  A lane remembers of each its token's number in the super tile (from bit
// 24) and the chunk's place in the token's row.
template <int DP>
struct Loader {
  using Ge = Geo4<DP>;
  uint32_t at[Ge::kBlocks];
  template <class A>
  __device__ __forceinline__ Loader(const A& a, const Columns& co, int wave) {
    const int lane = rare_lane();
    const uint32_t inv = (65535u + co.cpr) / (uint32_t)co.cpr;  // of numbers below 65,536 / cpr, which these are
#pragma unroll
    for (int j = 0; j < Ge::kBlocks; j++) {
      const int q = min((wave + j * Ge::kWaves) * 64 + lane, 32 * co.turn * co.cpr - 1);
      const int row = (int)(q * inv >> 16), c = q - row * co.cpr, r = row & 15;
      // a head's chunks change places where there are as many as the products take
      const int chunk = a.head_bytes == Ge::CH * 16 ? c ^ Ge::twist(r) : c;
      const int col = c < co.codes ? co.first * a.head_bytes + chunk * 16 : co.window + (c - co.codes) * 16;
      at[j] = (uint32_t)row << 24 | (uint32_t)col;
    }
  }

  // Issues the loads of the super tile at token t0 to the stage at LDS address `lds`.
  template <class A>
  __device__ __forceinline__ void load(const A& a, const Columns& co, const Pages& p, int wave, int t0, uint32_t lds) const {
    uint32_t to = lds + wave * 1024;
    asm volatile("" : "+s"(to));  // computed anew for each block: all of them are more than fits scalar registers
#pragma unroll
    for (int j = 0; j < Ge::kBlocks; j++) {
      if (wave + j * Ge::kWaves >= co.vat / 1024) break;
      uint32_t mine = at[j];
      asm volatile("" : "+v"(mine));  // nor are parts of it kept
      const uint64_t off = p.row_at(t0 + (int)(mine >> 24), a.page_bytes, a.row_bytes) + (mine & 0xFFFFFFu);
      load_lds(to + j * Ge::kWaves * 1024, a.k + off);
      load_lds(to + j * Ge::kWaves * 1024 + co.vat, a.v + off);
    }
  }
};

// Where a lane finds its part of a tile of one head, in bytes from the tile's first row.
// n = lane & 15, g = lane >> 4.
//   K: channels g DP / 4 .. of tokens n and 16 + n.
//   V: of tokens 4 g + i and 16 + 4 g + i the channels of column n of V^T's blocks, DP / 16 neighbours.
//      Where a head has the groups that the products take, a transposing read gives lane n
//      the scales of 4 tokens of group n % 4 (DP = 256: n % 8), and its channels are of that
//      group; elsewhere they are n DP / 16 .., and their scales are read one by one.
template <int DP>
struct Head {
  using Ge = Geo4<DP>;
  int kread, kscale, kstep, kmore, vread, vflip, vscale;
  int row;        // bytes of a row
  uint32_t bytes; // DP = 64: where the lane's channels of V are in their word
  int channel;    // the lane's first channel of V
  bool transposed;

  template <class A>
  __device__ __forceinline__ Head(const A& a, const Columns& co, int head) {
    const int lane = rare_lane(), n = lane & 15, g = lane >> 4;
    row = co.cpr * 16;
    const int codes = head * a.head_bytes, scales = co.codes * 16 + co.skew + 2 * head * a.groups;
    const bool full = a.head_bytes == Ge::CH * 16;
    const int last = a.head_bytes / 16 - 1;
    const int c = DP == 64 ? g >> 1 : DP == 128 ? g : 2 * g;
    // DP = 256: chunk c + 1 is at c's position ^ 1, or where the head has fewer the last again
    kread = n * row + codes + (full ? c ^ Ge::twist(n) : min(c, last)) * 16 + (DP == 64 ? (g & 1) * 8 : 0);
    kstep = DP == 256 ? (full ? (n * row + codes + ((c + 1) ^ Ge::twist(n)) * 16) : n * row + codes + min(c + 1, last) * 16) - kread : 0;
    kscale = n * row + scales + 2 * min(c, a.groups - 1);  // DP = 64: group g / 2 is chunk g / 2's
    kmore = c + 1 < a.groups ? 2 : 0;
    transposed = DP != 64 && full;
    const int group = DP == 128 ? n & 3 : (n >> 2 & 1) * 4 + (n & 3), j = DP == 128 ? n >> 2 : n >> 3;
    channel = transposed ? group * 32 + j * (DP / 16) : n * (DP / 16);
    const int word = min(channel / 8, a.head_bytes / 4 - (DP == 256 ? 2 : 1));  // what lies behind the head is nobody's
    // rows 4 g + i, i < 4, have one twist, for DP = 256 two
    const int first = full ? Ge::twist(4 * g) * 16 : 0, second = full ? Ge::twist(4 * g + 2) * 16 : 0;
    vread = 4 * g * row + codes + ((word * 4) ^ first);
    vflip = ((word * 4) ^ second) - ((word * 4) ^ first);
    bytes = 0x0C040C00u + (channel & 4 ? 0x00010001u : 0);
    vscale = transposed ? (4 * g + (n >> 2)) * row + scales + (DP == 256 ? (n & 1) * 8 : 0)
                        : 4 * g * row + scales + 2 * min(channel / 32, a.groups - 1);
  }
};

// Scores of a tile: S^T = K Q^T.
template <int DP, int RT>
__device__ __forceinline__ void scores(const Wave<DP, RT>& w, const Head<DP>& hd, const Nibbles& nb, const char* kt,
                                       f4 (&s)[RT][2]) {
  constexpr int KS = DP / 32;
#pragma unroll
  for (int r = 0; r < RT; r++) s[r][0] = s[r][1] = f4{0, 0, 0, 0};
#pragma unroll
  for (int sub = 0; sub < 2; sub++) {
    uint32_t k[KS];
    uint16_t ks[DP == 256 ? 2 : 1];
    const char* at = kt + sub * 16 * hd.row + hd.kread;
    if constexpr (DP == 64) {
      const uint2 x = *(const uint2*)at;
      k[0] = x.x;
      k[1] = x.y;
    } else {
#pragma unroll
      for (int j = 0; j < KS / 4; j++) {
        const u4 x = *(const u4*)(at + (j ? hd.kstep : 0));
#pragma unroll
        for (int e = 0; e < 4; e++) k[4 * j + e] = x[e];
      }
    }
    const char* sc = kt + sub * 16 * hd.row + hd.kscale;
    ks[0] = *(const uint16_t*)sc;
    if constexpr (DP == 256) ks[1] = *(const uint16_t*)(sc + hd.kmore);
    // fences for the scheduler, which else makes all numbers first and runs out of registers
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < KS; i++) {
      const h8 x = nb.numbers(k[i], both(ks[DP == 256 ? i / 4 : 0]));
#pragma unroll
      for (int r = 0; r < RT; r++) s[r][sub] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, w.q[r][i], s[r][sub], 0, 0, 0);
      if (i % 2) __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// Before the values of a tile of which some token does not exist or some query does not see
// some token: a number there that is not finite must not meet the zero weight of such a
// query.  In the stage, scales of tokens that do not exist become 0, and so do those that are
// no finite number, and codes whose number is none; returns whether there was such a number:
// add_odd() gives it to the queries that see it.
template <int DP, class A>
__device__ __forceinline__ bool clean_values(const A& a, const Columns& co, int head, char* vt, uint32_t alive) {
  const int lane = rare_lane(), tok = lane & 31;
  char* row = vt + tok * co.cpr * 16;
  uint16_t* scale = (uint16_t*)(row + co.codes * 16 + co.skew + 2 * head * a.groups);
  const int twist = a.head_bytes == Geo4<DP>::CH * 16 ? Geo4<DP>::twist(tok & 15) : 0;
  const bool there = (alive >> tok) & 1;
  bool found = false;
#pragma unroll 1
  for (int j = lane >> 5; j < a.groups; j += 2) {
    const uint16_t bits = scale[j], size = bits & 0x7FFF;
    if (there && size <= 0x6FFE) continue;  // 8 s is finite
    if (!there || size >= 0x7C00) {
      scale[j] = 0;
      found |= there;
      continue;
    }
    const float s = half_bits_to_float(bits);
    uint32_t* codes = (uint32_t*)(row + head * a.head_bytes + (j ^ twist) * 16);
#pragma unroll 1
    for (int i = 0; i < 32; i++) {
      const uint32_t w = codes[i / 8];
      const float x = (float)(_Float16)((float)((int)(w >> 4 * (i % 8) & 15) - 8) * s);
      if (x - x == 0.0f) continue;
      codes[i / 8] = (w & ~(15u << 4 * (i % 8))) | 8u << 4 * (i % 8);
      found = true;
    }
  }
  wait_lds();
  return __any(found);
}

// o += V^T P^T.  Row n of block b of V^T is channel b of the lane's, so that a lane's
// channels are neighbours in its word; its tokens come together two at a time.
// two: P^T + rest^T.
template <int DP, int RT>
__device__ __forceinline__ void values(Wave<DP, RT>& w, const Head<DP>& hd, const Nibbles& nb, const char* vt,
                                       const h8 (&p)[RT], bool two, const h8 (&rest)[RT]) {
  constexpr int VW = DP == 256 ? 2 : 1, HALVES = DP == 64 ? 1 : 2;  // words of a lane, halves of a word
  uint32_t x[8][VW];
  union { s4 t[2]; h2 s[4]; uint16_t u[8]; } sc;  // scales of tokens 4 g .. + 3, 16 + 4 g .. + 3
#pragma unroll
  for (int sub = 0; sub < 2; sub++) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const char* at = vt + (16 * sub + i) * hd.row + hd.vread + (DP == 256 && i >= 2 ? hd.vflip : 0);
      if constexpr (VW == 2) {
        const uint2 y = *(const uint2*)at;
        x[4 * sub + i][0] = y.x;
        x[4 * sub + i][1] = y.y;
      } else {
        x[4 * sub + i][0] = *(const uint32_t*)at;
      }
    }
  }
  int transposed = __builtin_amdgcn_readfirstlane(DP != 64 && hd.transposed);
  asm volatile("" : "+s"(transposed));  // one loop, not one for each case
  if (transposed) {
#pragma unroll
    for (int sub = 0; sub < 2; sub++)
      sc.t[sub] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(vt + 16 * sub * hd.row + hd.vscale));
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      sc.u[i] = *(const uint16_t*)(vt + (16 * (i >> 2) + (i & 3)) * hd.row + hd.vscale);
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int y = 0; y < 2 * VW * HALVES; y++) {  // 2 channels, of byte y / 2 % 2 or (odd y) 2 + that of words y / 4
    union { uint32_t u[4]; h8 h; } v[2];
#pragma unroll
    for (int j = 0; j < 4; j++) {  // tokens 4 g + 2 j, + 1 (j < 2), 16 + 4 g + 2 (j - 2), + 1
      const uint32_t w0 = x[2 * j][y / 2 / HALVES], w1 = x[2 * j + 1][y / 2 / HALVES];
      const uint32_t sel = (DP == 64 ? hd.bytes : 0x0C040C00u + (y / 2 & 1) * 0x00010001u) + (y & 1) * 0x00020002u;
      const uint32_t both = __builtin_amdgcn_perm(w1, w0, sel);
      v[0].u[j] = __builtin_bit_cast(uint32_t, nb.get<false>(both) * sc.s[j]);
      v[1].u[j] = __builtin_bit_cast(uint32_t, nb.get<true>(both) * sc.s[j]);
    }
#pragma unroll
    for (int b = 0; b < 2; b++) {
      const int block = y / 2 * 4 + 2 * b + (y & 1);
#pragma unroll
      for (int r = 0; r < RT; r++)
        w.o[r][block] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[b].h, p[r], w.o[r][block], 0, 0, 0);
      if (two)
#pragma unroll
        for (int r = 0; r < RT; r++)
          w.o[r][block] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[b].h, rest[r], w.o[r][block], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Scores of tokens that do not exist, or that a query does not see, become -inf.
template <int DP, int RT>
__device__ __forceinline__ void mask_scores(const QuantAttn& a, const Item& it, int row0, f4 (&s)[RT][2], int t0,
                                            uint32_t alive) {
  const int lane = rare_lane(), g = lane >> 4;
#pragma unroll
  for (int r = 0; r < RT; r++) {
    const int lim = row_lim(a, it, row0 + r * 16 + (lane & 15));
#pragma unroll
    for (int sub = 0; sub < 2; sub++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int tok = sub * 16 + 4 * g + i;
        s[r][sub][i] = ((alive >> tok) & 1) && t0 + tok < lim ? s[r][sub][i] : -__builtin_inff();
      }
  }
}

// ---------------------------------------------------------------------------
// One workgroup: a tile of rows against a split of the tokens
// ---------------------------------------------------------------------------
constexpr int kList = 512;  // table entries staged at a time
template <int DP>
struct QuantShared {
  static constexpr int kWaves = Geo4<DP>::kWaves;
  __attribute__((aligned(1024))) char stage[2][Geo4<DP>::kStage];  // then the sums of the waves
  int32_t list[kList];
  float m[kWaves][32], l[kWaves][32], scale[kWaves][32];
  uint32_t odd;  // clean_values() found something
  uint32_t bad;  // a page met so far is outside the pool
  int sums[kWaves], most[kWaves];
};
static_assert(sizeof(QuantShared<128>) <= 160 * 1024 / 2, "two workgroups a compute unit");

// The number of channel ch of kv head `head` in the row at p.
__device__ __forceinline__ float number_at(const QuantAttn& a, const char* p, int head, int ch) {
  const uint32_t w = *(const uint32_t*)(p + head * a.head_bytes + ch / 8 * 4);
  const _Float16 s = __builtin_bit_cast(_Float16, *(const uint16_t*)(p + a.scales + 2 * (head * a.groups + ch / 32)));
  const int e = ch % 8;
  return (float)((_Float16)(float)((int)((w >> (16 * (e & 1) + 4 * (e >> 1))) & 15) - 8) * s);
}

// After the sums of rows [row0, row1) are stored: what values() took out, for the rows that
// see it (a sum with such a number is an infinity or none whatever the weight, and stays
// so where the number was counted already).  Rare, and slow.  empty(head, row): of a
// direct item, whether nothing weighed anything for a row.
template <int kThreads, class A, class F>
__device__ __forceinline__ void add_odd(const A& a, const Item& it, const Span& span, int ranges, int row0, int row1,
                                        F empty) {
  const int tid = rare_thread();
  row1 = min(row1, it.rows);
#pragma unroll 1
  for (int range = 0; range < ranges; range++) {
    const Item cur = range_of(it, ranges, range);
    const Span sp = a.direct ? span_of(cur.lo, cur.hi, 0, 1, 1) : span;
    const int end = min(min(sp.to * kTile, cur.hi), row_lim(a, cur, row1 - 1));
#pragma unroll 1
    for (int t = max(sp.from * kTile, cur.lo); t < end; t++) {
      const int page = a.tables[(int64_t)cur.trow * a.B + (t >> a.shift)];
      if (page < 0 || page >= a.N) continue;
      const char* v = a.v + (uint64_t)(uint32_t)page * a.page_bytes + (uint64_t)(uint32_t)(t & (a.P - 1)) * a.row_bytes;
#pragma unroll 1
      for (int i = tid; i < it.heads * a.d; i += kThreads) {
        const int head = it.head + i / a.d, ch = i % a.d;
        const float x = number_at(a, v, head, ch);
        if (x - x == 0.0f) continue;
#pragma unroll 1
        for (int row = row0; row < row1; row++) {
          if (t >= row_lim(a, cur, row) || (a.direct && empty(head, row))) continue;
          if (a.direct) {
            uint16_t* to = out_at(a, it, head, row) + ch;
            *to = float_to_half_bits(half_bits_to_float(*to) + x);
          } else {
            a.part[part_at(a, it, head, row) * a.d + ch] += x;
          }
        }
      }
    }
    __syncthreads();
  }
}

// A wave holds all 16 RT rows of a row tile of its kv head and takes every turn-th tile of
// them; the waves share nothing but the super tiles until the end.  The next super tile is on its
// way while one is computed.
template <int DP, int RT>
__device__ __forceinline__ void run_few(const QuantAttn& a, const Item& it, const Span& span, QuantShared<DP>& sh) {
  using W = Wave<DP, RT>;
  constexpr int kWaves = Geo4<DP>::kWaves, kThreads = Geo4<DP>::kThreads;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ranges = ranges_of(a, it);
  const Columns co(a, it.head, it.heads);
  const int mine = wave / it.heads, hh = wave % it.heads;  // the wave's tile of a super tile, and its head
  const bool busy = mine < co.turn;
  const float c = log2_scale(a);
  const int row_tiles = (it.rows + 16 * RT - 1) / (16 * RT);
  const int list_tiles = (int)((int64_t)(kList - 1) * a.P / kTile) - 1;
  if (!a.direct && span.from >= span.to) return;
  const Span whole_span = a.direct ? span_of(it.lo, it.hi, 0, 1, 1) : span;
  const int span_from = whole_span.from, span_end = whole_span.to;
  const uint32_t lds = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char*)sh.stage[0]);

#pragma unroll 1
  for (int rt = it.row_tile; rt < row_tiles; rt += it.row_tiles) {
    // the first stretch's pages are on their way while what needs none of them is worked out
    int early = 0, early_base = -1;
    if (ranges == 1 && span_end > span_from) {
      early_base = span_from;
      const int b0 = max(span_from * kTile, it.lo) >> a.shift, b1 = (min(span_end * kTile, it.hi) - 1) >> a.shift;
      early = a.tables[(int64_t)it.trow * a.B + min(b0 + (int)threadIdx.x, b1)];
    }
    const Loader<DP> ld(a, co, wave);
    const Head<DP> hd(a, co, hh);
    const Nibbles nb;
    W w;
    w.clear();
    w.template load_queries<true>(a, it, it.head + hh, rt * 16 * RT, rare_lane());
    if (threadIdx.x == 0) sh.odd = sh.bad = 0;
#pragma unroll 1
    for (int range = 0; range < ranges; range++) {
      const Item cur = range_of(it, ranges, range);
      const Span sp = a.direct ? span_of(cur.lo, cur.hi, 0, 1, 1) : span;
      const int min_lim = row_lim(a, cur, rt * 16 * RT);
      // tiles behind this one nobody of these rows sees
      const int end = min(sp.to, (row_lim(a, cur, (rt + 1) * 16 * RT - 1) + kTile - 1) / kTile);
#pragma unroll 1
      for (int base = sp.from; base < end; base += list_tiles) {
        const int stop = min(base + list_tiles, end);
        const int b0 = max(base * kTile, cur.lo) >> a.shift, b1 = (min(stop * kTile, cur.hi) - 1) >> a.shift;
        __syncthreads();  // the list and the stages are free
        for (int i = rare_thread(); i <= b1 - b0; i += kThreads) {
          const int page = early_base == base && i < kThreads ? early : a.tables[(int64_t)cur.trow * a.B + b0 + i];
          const bool ok = page >= 0 && page < a.N;
          sh.list[i] = ok ? page : -1;
          if (!ok) sh.bad = 1;
        }
        __syncthreads();
        // tokens that exist for this stretch lie in its blocks
        const bool bad = __builtin_amdgcn_readfirstlane(sh.bad) != 0;
        const Pages pages{sh.list, b0, max(base * kTile, cur.lo), min(stop * kTile, cur.hi), a.shift, a.P - 1};
        const int limit = busy ? stop : 0, whole_lo = bad ? 0x7FFFFFFF : pages.lo;
        int slot = 0;
        ld.load(a, co, pages, wave, base * kTile, lds);
        // The queries are here before the loop: the compiler would wait for them in each step, and
        // with them for all loads under way.
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
          for (int ks = 0; ks < W::KS; ks++) asm volatile("" : "+v"(w.q[r][ks]));
#pragma unroll 1
        for (int at = base; at < stop; at += co.turn, slot ^= 1) {
          wait_loads<0>();
          wait_lds();
          __builtin_amdgcn_s_barrier();  // the super tile is there, and the other stage has been read
          asm volatile("" ::: "memory");
          if (at + co.turn < stop)
            ld.load(a, co, pages, wave, (at + co.turn) * kTile, lds + (slot ^ 1) * Geo4<DP>::kStage);
          const int tile = at + mine;
          if (tile < limit) {
            const char* kt = sh.stage[slot] + mine * 512 * co.cpr;
            char* vt = sh.stage[slot] + co.vat + mine * 512 * co.cpr;
            const bool whole = tile * kTile >= whole_lo && (tile + 1) * kTile <= pages.hi;
            const uint32_t alive = whole ? 0xFFFFFFFFu : find(pages, tile * kTile);
            f4 s[RT][2];
            h8 p[RT];
            float mx[RT];
            scores(w, hd, nb, kt, s);
            const bool all = alive == 0xFFFFFFFFu && (tile + 1) * kTile <= min_lim;
            if (!all) mask_scores<DP, RT>(a, cur, rt * 16 * RT, s, tile * kTile, alive);
            const bool raise = w.peaks(s, c, mx);
            w.reference(raise, mx, c);
            w.weights(s, c, p);
            if (!all && clean_values<DP>(a, co, hh, vt, alive)) sh.odd = 1;
            // A workgroup alone with a few tokens, whose weights' roundings do not average out and whose time
            // is not in its products, gives the second product the weights in two parts.
            h8 rest[RT];
            if (a.direct) w.rests(s, c, p, rest);
            values(w, hd, nb, vt, p, a.direct, rest);
          }
          asm volatile("" ::: "memory");  // one end of the loop's body, not two loops
        }
      }
    }
    const int tid = rare_thread(), n = tid & 15, g = (tid & 63) >> 4;
    __syncthreads();  // the stages are free, and bad is known
    if (sh.bad && tid == 0) atomicOr(a.status, kBadPage);
    const int row0 = rt * 16 * RT, rows = min(it.rows - row0, 16 * RT);
    // A lane has row n of 16, and of each row 4 g + i of a block of results the channel of lane 4 g + i.
    auto quad_of = [&](int r, int b, int i) {
      return r == 0 ? f4{w.o[0][b][i], w.o[0][b + 1][i], w.o[0][b + 2][i], w.o[0][b + 3][i]}
                    : f4{w.o[RT - 1][b][i], w.o[RT - 1][b + 1][i], w.o[RT - 1][b + 2][i], w.o[RT - 1][b + 3][i]};
    };
    auto store = [&](int h, int row, int ch, f4 x) {
      if (a.direct) store_out(out_at(a, it, it.head + h, row0 + row) + ch, quotient_of(x, sh.m[h][row]));
      else *(f4*)(a.part + part_at(a, it, it.head + h, row0 + row) * a.d + ch) = x;
    };
    auto store_sums = [&](int h, int row, float m, float l) {
      if (a.direct) {
        sh.m[h][row] = l == 0.0f ? 0.0f : 1.0f / l;
        if (row < rows && a.lse) *lse_at(a, it, it.head + h, row0 + row) = lse_of(m, l);
      } else if (row < rows) {
        const int64_t at = part_at(a, it, it.head + h, row0 + row);
        *(float2*)(a.ml + 2 * at) = float2{m, l};
      }
    };
    if (co.turn == 1) {  // a wave has all of its head's sums
      if (busy) {
#pragma unroll
        for (int r = 0; r < RT; r++) {
          const float l = w.sum(r);
          if (g == 0) store_sums(hh, r * 16 + n, w.m[r], l);
        }
        wait_lds();
#pragma unroll 1
        for (int r = 0; r < RT; r++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int ch = __shfl(hd.channel, 4 * g + i);
#pragma unroll
            for (int b = 0; b < W::NB; b += 4)
              if (r * 16 + n < rows && ch + b < a.d) store(hh, r * 16 + n, ch + b, quad_of(r, b, i));
          }
      }
    } else {
      // The waves' sums together, against the largest reference exponent.  Loops over the waves are
      // unrolled, so that their reads are under way together.
      constexpr int kQuads = DP / 4;  // of a row, rotated by row
      static_assert(sizeof(sh.stage) >= (size_t)kWaves * 16 * kQuads * 16, "room for the sums");
      f4* sums = (f4*)sh.stage;
      auto put = [&](int r) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int ch = __shfl(hd.channel, 4 * g + i);
#pragma unroll
          for (int b = 0; b < W::NB; b += 4)
            if (r * 16 + n < rows) sums[(wave * 16 + n) * kQuads + (((ch + b) / 4 + n) & (kQuads - 1))] = quad_of(r, b, i);
        }
      };
#pragma unroll
      for (int r = 0; r < RT; r++) {
        const float l = w.sum(r);
        if (g == 0) {
          sh.m[wave][r * 16 + n] = w.m[r];
          sh.l[wave][r * 16 + n] = l;
        }
      }
      put(0);
      __syncthreads();
      auto wave_of = [&](int h, int y) { return h + it.heads * min(y, co.turn - 1); };  // that has tile y of head h
      if (tid < 16 * RT * it.heads) {
        const int x = tid % (16 * RT), h = tid / (16 * RT);
        float m = -__builtin_inff(), l = 0.0f, ms[kWaves], ls[kWaves];
#pragma unroll
        for (int y = 0; y < kWaves; y++) {
          ms[y] = sh.m[wave_of(h, y)][x];
          ls[y] = sh.l[wave_of(h, y)][x];
        }
#pragma unroll
        for (int y = 0; y < kWaves; y++) m = fmaxf(m, ms[y]);
#pragma unroll
        for (int y = 0; y < kWaves; y++) {
          // a wave without a reference has weighed nothing, or only what is no number
          const float f = ms[y] == m ? 1.0f : ms[y] == -__builtin_inff() && ls[y] != 0.0f
                                 ? 1.0f : __builtin_amdgcn_exp2f(ms[y] - m);
          sh.scale[wave_of(h, y)][x] = f;
          l += y < co.turn ? f * ls[y] : 0.0f;
        }
        store_sums(h, x, m, l);
      }
#pragma unroll 1
      for (int r = 0; r * 16 < rows; r++) {
        if (r) {
          __syncthreads();
          put(r);
        }
        __syncthreads();
        const int here = rows - r * 16;
#pragma unroll 1
        for (int i = tid; i < it.heads * 16 * kQuads; i += kThreads) {
          const int quad = i % kQuads, x = i / kQuads % 16, h = i / (16 * kQuads), row = r * 16 + x;
          if (quad * 4 >= a.d || x >= here) continue;
          f4 part[kWaves], sum{0, 0, 0, 0};
          float f[kWaves];
#pragma unroll
          for (int y = 0; y < kWaves; y++) {
            const int from = wave_of(h, y);
            f[y] = sh.scale[from][row];
            part[y] = sums[(from * 16 + x) * kQuads + ((quad + x) & (kQuads - 1))];
          }
#pragma unroll
          for (int y = 0; y < kWaves; y++)
            if (y < co.turn) sum += f[y] * part[y];
          store(h, row, quad * 4, sum);
        }
      }
    }
    __syncthreads();
    if (sh.odd)
      add_odd<kThreads>(a, it, span, ranges, row0, row0 + 16 * RT,
                        [&](int h, int row) { return sh.m[h - it.head][row - row0] == 0.0f; });
    __syncthreads();  // m, l, scale and the sums are free
  }
}

// Many rows of one head: a wave holds 16 RT of the 16 RT kWaves, and all waves read the same
// tiles, whose numbers they make once, as binary16 in the form that cg_attention.h's products
// take.  Codes come to registers two tiles ahead, numbers are made one tile ahead of their products,
// and one barrier a tile publishes them and frees the tile before.
template <int DP, int RT>
__device__ __forceinline__ void run_many(const QuantAttn& a, const Item& it, const Span& span, QuantShared<DP>& sh) {
  using W = Wave<DP, RT>;
  constexpr int kWaves = Geo4<DP>::kWaves, kThreads = Geo4<DP>::kThreads;
  constexpr int CH = DP / 8;  // 8-channel words of a row
  constexpr int kSides = DP == 64 ? 1 : 2, kTokens = 64 * CH / kThreads / kSides;
  constexpr int kTileBytes = Geo<DP>::BYTES;
  static_assert(sizeof(sh.stage) >= 4 * kTileBytes && kTokens * kSides * kThreads == 64 * CH, "two tiles of K and V");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ranges = ranges_of(a, it);
  const float c = log2_scale(a);
  const int tile_rows = 16 * RT * kWaves, row_tiles = (it.rows + tile_rows - 1) / tile_rows;
  const int list_tiles = (int)((int64_t)(kList - 1) * a.P / kTile) - 1;
  if (!a.direct && span.from >= span.to) return;
  char* tiles = sh.stage[0];  // K, V, K, V
  const int token0 = threadIdx.x / CH % 32;
  const bool side0 = threadIdx.x >= 32 * CH;  // DP = 64: V

#pragma unroll 1
  for (int rt = it.row_tile; rt < row_tiles; rt += it.row_tiles) {
    const int row0 = rt * tile_rows + wave * 16 * RT;
    const Nibbles nb;
    const Places<DP> at_lane;
    W w;
    w.clear();
    w.load_queries(a, it, it.head, row0, rare_lane());
    if (threadIdx.x == 0) sh.odd = sh.bad = 0;
#pragma unroll 1
    for (int range = 0; range < ranges; range++) {
      const Item cur = range_of(it, ranges, range);
      const Span sp = a.direct ? span_of(cur.lo, cur.hi, 0, 1, 1) : span;
      const int min_lim = __builtin_amdgcn_readfirstlane(row_lim(a, cur, rt * tile_rows));
      const int end = __builtin_amdgcn_readfirstlane(min(sp.to, (row_lim(a, cur, (rt + 1) * tile_rows - 1) + kTile - 1) / kTile));
#pragma unroll 1
      for (int base = __builtin_amdgcn_readfirstlane(sp.from); base < end; base += list_tiles) {
        const int stop = min(base + list_tiles, end);
        const int b0 = max(base * kTile, cur.lo) >> a.shift, b1 = (min(stop * kTile, cur.hi) - 1) >> a.shift;
        __syncthreads();  // the list and the tiles are free
        for (int i = rare_thread(); i <= b1 - b0; i += kThreads) {
          const int page = a.tables[(int64_t)cur.trow * a.B + b0 + i];
          const bool ok = page >= 0 && page < a.N;
          sh.list[i] = ok ? page : -1;
          if (!ok) sh.bad = 1;
        }
        __syncthreads();
        const bool bad = __builtin_amdgcn_readfirstlane(sh.bad) != 0;
        const Pages pages{sh.list, b0, __builtin_amdgcn_readfirstlane(max(base * kTile, cur.lo)), __builtin_amdgcn_readfirstlane(min(stop * kTile, cur.hi)), a.shift, a.P - 1};
        auto whole = [&](int tile) { return !bad && tile * kTile >= pages.lo && (tile + 1) * kTile <= pages.hi; };
        // This thread's words: of kTokens tokens, kThreads / CH apart, of K and of V (DP = 64: of one of them).
        uint32_t word[kTokens][kSides];
        uint16_t scale[kTokens][kSides];
        auto fetch = [&](int tile) {
          const int chunk = threadIdx.x % CH;
          const int code = it.head * a.head_bytes + min(chunk * 4, a.head_bytes - 4);
          const int at = a.scales + 2 * (it.head * a.groups + min(chunk / 4, a.groups - 1));
#pragma unroll
          for (int i = 0; i < kTokens; i++) {
            const uint64_t row = pages.row_at(tile * kTile + token0 + i * (kThreads / CH), a.page_bytes, a.row_bytes);
#pragma unroll
            for (int v = 0; v < kSides; v++) {
              const char* p = (DP == 64 ? side0 : v != 0) ? a.v + row : a.k + row;
              word[i][v] = *(const uint32_t*)(p + code);
              scale[i][v] = *(const uint16_t*)(p + at);
            }
          }
        };
        // all: every query sees every token of the tile
        auto make = [&](int tile, bool all, int to) {
          const uint32_t alive = whole(tile) ? 0xFFFFFFFFu : find(pages, tile * kTile);
          const int chunk = threadIdx.x % CH;
#pragma unroll
          for (int i = 0; i < kTokens; i++)
#pragma unroll
            for (int y = 0; y < kSides; y++) {
              const int tok = token0 + i * (kThreads / CH);
              const bool v = DP == 64 ? side0 : y != 0, there = ((alive >> tok) & 1) && chunk * 8 < a.d;
              u4 x = __builtin_bit_cast(u4, nb.numbers(word[i][y], both(scale[i][y])));
              if (!there) x = u4{0, 0, 0, 0};
              if (!all && v) {
                // a number that is not finite must not meet the zero weight of a query that does not see
                // it: add_odd() gives it to those that do
                bool odd = false;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                  const uint32_t keep = ((x[j] & 0x7C00u) == 0x7C00u ? 0 : 0xFFFFu) | ((x[j] & 0x7C000000u) == 0x7C000000u ? 0 : 0xFFFF0000u);
                  odd |= keep != 0xFFFFFFFFu;
                  x[j] &= keep;
                }
                if (odd) sh.odd = 1;
              }
              *(u4*)(tiles + (2 * to + v) * kTileBytes + tok * DP * 2 + (chunk ^ swizzle<DP>(tok)) * 16) = x;
            }
        };
        auto seen = [&](int tile) { return whole(tile) && (tile + 1) * kTile <= min_lim; };
        int slot = 0;
        fetch(base);
        make(base, seen(base), 0);
        if (base + 1 < stop) fetch(base + 1);
#pragma unroll 1
        for (int tile = base; tile < stop; tile++, slot ^= 1) {
          wait_lds();
          __builtin_amdgcn_s_barrier();  // the tile is there, and the other one has been read
          asm volatile("" ::: "memory");
          if (tile + 1 < stop) make(tile + 1, seen(tile + 1), slot ^ 1);
          if (tile + 2 < stop) fetch(tile + 2);
          if (row0 < it.rows) {
            const char *kt = tiles + 2 * slot * kTileBytes, *vt = kt + kTileBytes;
            f4 s[RT][2];
            h8 p[RT];
            float mx[RT];
            w.scores(kt, at_lane.fresh(), s, [] {});
            if (!seen(tile))
              mask_scores<DP, RT>(a, cur, row0, s, tile * kTile, whole(tile) ? 0xFFFFFFFFu : find(pages, tile * kTile));
            const bool raise = w.peaks(s, c, mx);
            w.reference(raise, mx, c);
            w.weights(s, c, p);
            w.values(vt, at_lane.fresh(), p, [] {});
          }
          asm volatile("" ::: "memory");  // one end of the loop's body, not two loops
        }
      }
    }
    const int tid = rare_thread(), n = tid & 15, g = (tid & 63) >> 4;
    __syncthreads();
    if (sh.bad && tid == 0) atomicOr(a.status, kBadPage);
#pragma unroll
    for (int r = 0; r < RT; r++) {
      const float l = w.sum(r);
      const int row = row0 + r * 16 + n;
      if (row >= it.rows) continue;
      if (a.direct) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t* to = out_at(a, it, it.head, row);
#pragma unroll
        for (int b = 0; b < W::NB; b++)
          if (b * 16 + g * 4 < a.d) store_out(to + b * 16 + g * 4, quotient_of(w.o[r][b], inv));
        if (g == 0) sh.m[wave][r * 16 + n] = inv;
        if (g == 0 && a.lse) *lse_at(a, it, it.head, row) = lse_of(w.m[r], l);
        continue;
      }
      const int64_t at = part_at(a, it, it.head, row);
      if (g == 0) *(float2*)(a.ml + 2 * at) = float2{w.m[r], l};
#pragma unroll
      for (int b = 0; b < W::NB; b++)
        if (b * 16 + g * 4 < a.d) *(f4*)(a.part + at * a.d + b * 16 + g * 4) = w.o[r][b];
    }
    __syncthreads();
    if (sh.odd)
      add_odd<kThreads>(a, it, span, ranges, rt * tile_rows, (rt + 1) * tile_rows, [&](int, int row) {
        return sh.m[(row - rt * tile_rows) / (16 * RT)][row % (16 * RT)] == 0.0f;
      });
    __syncthreads();  // m, the list and the tiles are free
  }
}

// Tiles of sequence s's own tokens, 0 without queries.
__device__ __forceinline__ int tiles_of(const QuantAttn& a, int s) {
  const int row = row_of(a, s);
  const bool in = row >= 0 && row < a.R;
  const int len = a.lens[in ? row : 0], m = queries_of(a.q_starts[s], a.q_starts[s + 1], a.n_q);
  int pre = 0;
  if (a.n_groups) {  // the last group that begins at or before s
    int lo = -1, hi = a.n_groups;
    while (hi - lo > 1) {
      const int at = (lo + hi) >> 1;
      if (a.group_starts[at] <= s) lo = at; else hi = at;
    }
    if (lo >= 0 && s < a.group_starts[lo + 1]) pre = max(a.prefix_lens[lo], 0);
  }
  return in && m > 0 && len_ok(a, len) && len > pre ? (len + kTile - 1) / kTile - pre / kTile : 0;
}

// The tiles of each sequence's own tokens, added up: at[s] before sequence s, at[n_seqs] in all.  Returns
// how many are a part.
// (Cut into splits of one length the last of them run when most are done, and the chip's
// dispatcher does not fill all slots evenly: 64 sequences of 1,000 to 9,216 tokens
// took 123 to 136 us.)
__device__ __forceinline__ int add_up(const QuantAttn& a, int* at, int* sums, int* most) {
  const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x / 64;
  const int mine = (a.n_seqs + blockDim.x - 1) / blockDim.x, s0 = min(tid * mine, a.n_seqs), s1 = min(s0 + mine, a.n_seqs);
  int sum = 0, top = 0;
#pragma unroll 1
  for (int s = s0; s < s1; s++) {
    const int n = tiles_of(a, s);
    at[s] = sum;
    sum += n;
    top = max(top, n);
  }
  int before = sum;
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) {
    const int x = __shfl_up(before, i);
    top = max(top, __shfl_xor(top, i));
    if (lane >= i) before += x;
  }
  if (lane == 63) {
    sums[tid >> 6] = before;
    most[tid >> 6] = top;
  }
  __syncthreads();
  before -= sum;
  int all = 0;
  top = 0;
#pragma unroll 1
  for (int w = 0; w < waves; w++) {
    if (w < tid >> 6) before += sums[w];
    all += sums[w];
    top = max(top, most[w]);
  }
#pragma unroll 1
  for (int s = s0; s < s1; s++) at[s] += before;
  if (tid == 0) at[a.n_seqs] = all;
  __syncthreads();
  all = __builtin_amdgcn_readfirstlane(all);
  top = __builtin_amdgcn_readfirstlane(top);
  return tiles_of_part(all, top, a.parts, a.rest_splits, a.rest_least);
}

// What a workgroup computes next: items of the launch, or its part of the sequences' own tokens,
// for one row tile of theirs and its kv heads.
struct Work {
  int part, per, base, pos, end;  // tiles, of the sequences' behind one another: base where sequence s begins
  int s, w;                       // the next sequence, or item
  bool parts;
};

template <int DP, int MODE>
__device__ __forceinline__ void run_item(const QuantAttn& a, const Item& it, const Span& span, QuantShared<DP>& sh) {
  if constexpr (is_many(MODE)) run_many<DP, tiles_of_rows(MODE)>(a, it, span, sh);
  else run_few<DP, tiles_of_rows(MODE)>(a, it, span, sh);
}

template <int DP, int PRE, int REST, int CUT>
__global__ __launch_bounds__(Geo4<DP>::kThreads, resident4(PRE, REST) * Geo4<DP>::kWaves / 4) void k_quant_attention(
    QuantAttn a, int end) {
  __shared__ QuantShared<DP> sh;
  a.direct = CUT == kAlone;
  if constexpr (CUT != kParts) a.parts = 0;
  if constexpr (CUT == kAlone) {
    a.pre_groups = a.pre_splits = 0;
    a.rest_splits = a.rest_heads = a.pre_heads = a.pre_least = a.rest_least = 1;
  }
  const int columns = a.kv / a.rest_heads, pre_items = a.pre_groups * a.pre_splits * a.pre_tiles * (a.kv / a.pre_heads);
  Item it;
  Work wk{0, 1, 0, 0, 0, 0, (int)blockIdx.x, CUT == kParts && (int)blockIdx.x >= pre_items};
  if (wk.parts) {
    static_assert(sizeof(sh.stage) >= (kMostListed + 1) * 4, "room for the sums of tiles");
    int* at = (int*)sh.stage;
    wk.per = add_up(a, at, sh.sums, sh.most);
    uint32_t w = wk.w - pre_items;
    it.heads = a.rest_heads;
    it.head = w % columns * a.rest_heads;
    w /= columns;
    it.row_tile = w % a.rest_tiles;
    wk.part = w / a.rest_tiles;
    const int all = __builtin_amdgcn_readfirstlane(at[a.n_seqs]);
    wk.pos = (int)min((int64_t)wk.part * wk.per, (int64_t)all);
    wk.end = min(wk.pos + wk.per, all);
    if (it.head == 0 && it.row_tile == 0)  // sequences without tiles of their own have no other workgroup
#pragma unroll 1
      for (int s = wk.part; s < a.n_seqs; s += a.parts) {
        if (__builtin_amdgcn_readfirstlane(at[s + 1] - at[s]) != 0) continue;
        it.split = 0;
        rest_item(a, s, it);
        say_used(a, it, split_of(0, it.pre, a.pre_splits, a.pre_least).used, 0);
      }
    int s = -1;  // the last sequence that begins at or before the part
    for (int hi = a.n_seqs; hi - s > 1;) {
      const int m = (s + hi) >> 1;
      if (__builtin_amdgcn_readfirstlane(at[m]) <= wk.pos) s = m; else hi = m;
    }
    wk.s = s;
    wk.base = __builtin_amdgcn_readfirstlane(at[s]);  // the stages take the place of the sums from here
  }
#pragma unroll 1
  while (wk.parts ? wk.pos < wk.end && wk.s < a.n_seqs : wk.w < end) {
    Span span{0, 0};
    bool go, prefix = false;
    int own = -1;  // splits of the sequence's own tokens
    if (wk.parts) {
      const int s = wk.s++, tiles = tiles_of(a, s);
      if (tiles == 0) continue;
      const Parts in = parts_of(wk.base, tiles, wk.per);
      const int from = wk.pos - wk.base, n = min(tiles - from, wk.end - wk.pos);
      it.split = wk.part - in.first;
      go = rest_item(a, s, it);
      own = in.used;
      if (go) span = Span{it.lo / kTile + from, it.lo / kTile + from + n};
      wk.pos += n;
      wk.base += tiles;
    } else {
      go = item_of(a, wk.w, it);
      prefix = wk.w < pre_items;
      if (go) span = prefix ? span_of(0, it.hi, it.split, a.pre_splits, a.pre_least)
                                      : span_of(it.lo, it.hi, it.split, a.rest_splits, a.rest_least);
      wk.w += gridDim.x;
    }
    if (go) {
      if (PRE == REST || !prefix) run_item<DP, REST>(a, it, span, sh);
      else run_item<DP, PRE>(a, it, span, sh);
    }
    if (a.direct) {
      if (!it.ok) refuse(a, it);
    } else if (it.says) {
      say_used(a, it, split_of(0, it.pre, a.pre_splits, a.pre_least).used,
               own < 0 ? split_of(it.pre, it.hi, a.rest_splits, a.rest_least).used : own);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// The kernel of the call's modes and cut, if it is built.
template <int DP, int I = 0>
bool launch(int pre, int rest, int cut, const QuantAttn& a, int64_t items, hipStream_t st) {
  constexpr int PRE = I / kCuts / kModes, REST = I / kCuts % kModes, CUT = I % kCuts;
  if constexpr (PRE == kModes) {
    return false;
  } else {
    if constexpr (built(DP, PRE, REST, CUT)) {
      if (pre == PRE && rest == REST && cut == CUT) {
        const int grid = (int)std::min<int64_t>(items, 1 << 22);
        if (items > 0) k_quant_attention<DP, PRE, REST, CUT><<<grid, Geo4<DP>::kThreads, 0, st>>>(a, (int)items);
        return true;
      }
    }
    return launch<DP, I + 1>(pre, rest, cut, a, items, st);
  }
}
bool launch(const Plan& p, const QuantAttn& a, int64_t items, hipStream_t st) {
  return p.dp == 64    ? launch<64>(p.pre_mode, p.rest_mode, p.cut(), a, items, st)
         : p.dp == 128 ? launch<128>(p.pre_mode, p.rest_mode, p.cut(), a, items, st)
                       : launch<256>(p.pre_mode, p.rest_mode, p.cut(), a, items, st);
}

}  // namespace
}  // namespace cg

using namespace cg;

extern "C" {

int cg_quant_attention_workspace(const cg_paged_cache* c, const cg_quant_form* f, const cg_attention* a, size_t* bytes) {
  if (int rc = check_quant_attention(c, f, a)) return rc;
  if (!bytes) return fail(CG_E_INVAL, "bytes is NULL");
  *bytes = (4 * plan_of(*c, *f, *a).words + 15) & ~(size_t)15;
  return CG_OK;
}

int cg_quant_attention_async(const cg_paged_cache* c, const cg_quant_form* f, const cg_attention* a,
                             void* workspace_dev, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  if (int rc = cg_quant_attention_workspace(c, f, a, &need)) return rc;
  if (int rc = check_attention_strides(a)) return rc;
  if (a->n_seqs == 0 || a->n_q == 0) return CG_OK;
  if (int rc = check_attention_memory(c, a, workspace_dev, workspace_bytes, need)) return rc;
  DeviceGuard dg(c->device);
  if (!dg.ok) return fail(CG_E_HIP, "cannot select the cache's device");
  const Plan p = plan_of(*c, *f, *a);
  const QuantRow r = quant_row(*f);
  QuantAttn v{view(*c, *a, f->channels), r.head, r.groups, r.scales, (uint32_t)r.row,
              (uint32_t)r.row * (uint32_t)c->page_tokens, p.pre_least, p.rest_least, p.turn, p.pre_heads, p.direct, p.parts};
  const int64_t layer = (int64_t)a->layer * c->num_pages * v.page_bytes;
  v.k = (const char*)c->k_pool_dev + layer;
  v.v = (const char*)c->v_pool_dev + layer;
  v.pre_splits = p.pre_splits;
  v.rest_splits = p.rest_splits;
  v.pre_tiles = p.pre_tiles;
  v.rest_tiles = p.rest_tiles;
  v.rest_heads = p.rest_heads;
  v.pre_groups = p.pre_groups;
  v.part = (float*)workspace_dev;
  v.ml = v.part + (size_t)(p.pre_splits + p.rest_splits) * a->n_q * a->n_heads * a->head_dim;
  v.used = (int32_t*)(v.ml + (size_t)2 * (p.pre_splits + p.rest_splits) * a->n_q * a->n_heads);
  const int64_t pre = (int64_t)p.pre_groups * p.pre_splits * p.pre_tiles * (v.kv / p.pre_heads);
  const int64_t rest = (int64_t)(p.parts ? p.parts : a->n_seqs * (int64_t)p.rest_splits) * p.rest_tiles * (v.kv / p.rest_heads);
  hipStream_t st = (hipStream_t)stream;
  if (!launch(p, v, pre + rest, st)) return fail(CG_E_HIP, "attention over 4 bits: no kernel for the call's rows");
  if (!p.direct) {
    const int total = p.pre_splits + p.rest_splits;
    v.join = std::min(total <= 2 ? 1 : total <= 8 ? 2 : 8, kThreads / (v.d / 4));
    const int heads = kThreads / (v.d / 4) / v.join;
    k_join<<<dim3(a->n_q, (v.H + heads - 1) / heads), kThreads, 0, st>>>(v);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? CG_OK : hip_fail(e, "attention over 4 bits");
}

}  // extern "C"
