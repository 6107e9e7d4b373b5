// Attention of new tokens over a paged cache whose groups of sequences share a
// prefix (include/cachegen.h, cg_attention_prefix_async).
//
// With s_t = c (q . k_t), c = scale log2(e), a workgroup computes for its rows (query,
// head) and its tokens T the sums l = sum_T 2^(s_t - m) and o = sum_T 2^(s_t - m) v_t
// against a reference exponent m that follows the largest score.  Sums against
// different m join by factors 2^(m - m'), so any split of the tokens will do: a
// prefix's rows are those of all sequences of the group, which is what reads the prefix
// once; a sequence's own tokens are computed for its rows alone; long stretches are
// dealt to several workgroups.  k_join adds up and divides.  l, o and m are
// binary32; the weights 2^(s_t - m) are rounded to binary16 (a relative 2^-11 each) for
// the product with v, after they went into l, which lse takes unrounded.
//
// Bounds: reading every token of K and V once, or the products.  Measured, k_attention
// and k_join, the call repeated (and with other data in the caches in between): 64
// requests of 32 heads (8 of K and V, 128 channels) on 9,216 shared and up to 600 own
// tokens, 122 MB and 10 GFLOP, in 35 + 7 us (50): the tail of the sequences' own tokens
// and the join's reading back of the sums are what is left above the 26 us of a copy of
// these bytes.  21 requests of 32 heads, each with its K and V, 121 MB, in 29 + 5 us
// (37).  32 requests of 64 heads on 81,920 shared tokens, 366 MB and 86 GFLOP, in 115 + 10
// us at least (128; 137 when repeated without a pause, as power then allows): 0.75 PFLOP/s
// against 1.3 of a large library product; the matrix units are busy for 39% of the time and
// share the issue slots with the exponentials (about as many vector cycles as products).
#include <algorithm>
#include <type_traits>

#include "cg_hostapi.h"
#include "cg_internal.h"
#include "cg_paged.h"
#include "cg_ranges.h"

namespace cg {
namespace {

constexpr uint32_t kBadPage = 2u, kRefused = 4u;  // status bits

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s4 lds_s4;

constexpr int kThreads = 256;    // of a joining workgroup
// Tiles of a split of shared prefixes that take all of the chip's slots and leave the rest
// to wait for them: with fewer, half of the slots are the faster choice (14 requests of
// 64 heads, 32 of K and V, on 2,005 shared tokens: 30 us with half, 34 with all).
constexpr int kLong = 32;
// Weights are 2^(score - m) with m at most kSlack above what the running maximum
// was when it was last raised, and kLift below it: up to 2^14, and binary16's
// normal range reaches down to 2^-20 of the largest.
constexpr float kSlack = 8.0f, kLift = 6.0f;

struct Attn {
  int C, P, shift, N, R, B;
  const char *k, *v;  // the layer's pools
  const int32_t *tables, *lens;
  uint32_t* status;
  int H, G, d, kv;  // query heads, heads per kv head, head dimension, kv heads
  float scale;
  int n_seqs, n_q, n_groups;
  const int32_t *rows, *q_starts, *group_starts, *prefix_lens;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t q_stride, out_stride;
  // the launch: splits of a prefix and of a sequence's rest, row tiles that have
  // workgroups of their own (there may be more)
  int pre_splits, rest_splits, pre_tiles, rest_tiles, pre_groups, join;
  int rest_heads;  // kv heads of a workgroup that deals out the rest's tokens: 1, 2 or 4
  float* part;  // [pre_splits + rest_splits][n_q][H][d] sums, not divided
  float* ml;    // the same with [2]: reference exponent m, sum of weights l
  // [n_q]: splits of the prefix and (in the upper half) of the rest that the query's
  // sums are in, -1 if its sequence is refused; of queries that have a sequence
  int32_t* used;
};

// The same for kernels in which one item has all of its queries' tokens (the
// prefix's, unshared, and then the rest's), writes the outputs itself and nothing is
// joined.  Their own kernels: the tests for it cost the others 5%.
template <bool kDirect>
struct Call : Attn {
  static constexpr bool direct = kDirect;
};

// Largest i in [0, n) with a[i] <= x, or -1, a ascending; every lane of the wave
// gets it.  64 samples a step: one round of loads up to n = 64, two up to 4,096.
__device__ __forceinline__ int last_at_most(const int32_t* a, int n, int x) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = n;  // the answer is in [lo - 1, lo + len - 1]
  while (len > 0) {
    const int step = (len + 63) >> 6;
    const int i = lane * step;
    const uint64_t hit = __ballot(i < len && a[lo + (i < len ? i : 0)] <= x);
    const int n_hit = __popcll(hit);
    if (n_hit == 0) return lo - 1;
    const int at = (n_hit - 1) * step;  // a[lo + at] <= x, and not the next sample
    len = min(step, len - at) - 1;
    lo += at + 1;
  }
  return lo - 1;
}

__device__ __forceinline__ int row_of(const Attn& a, int s) { return a.rows ? a.rows[s] : s; }
__device__ __forceinline__ bool len_ok(const Attn& a, int64_t n) {
  return n >= 0 && n <= (int64_t)a.B << a.shift;
}

struct Seq {
  bool ok;           // its row, length, queries and prefix fit together
  int row, len, pre; // table row, tokens, those of the shared prefix
  int q0, m;         // first query, queries
  int first;         // the group's first sequence, -1 if it has no prefix
};

// Sequence s; all of it is uniform over the wave.  Loads that do not need one
// another are issued together, the groups' (up to 63) by the lanes: what a workgroup
// does before its first token is a chain of latencies.
__device__ __forceinline__ Seq sequence(const Attn& a, int s) {
  Seq q;
  q.row = row_of(a, s);
  q.q0 = a.q_starts[s];
  const int end = a.q_starts[s + 1];
  int g = -1, start = 0, next = 0, pre = 0;
  if (a.n_groups > 0 && a.n_groups < 64) {
    const int lane = threadIdx.x & 63;
    const int gs = a.group_starts[min(lane, a.n_groups)];
    const int pl = a.prefix_lens[min(lane, a.n_groups - 1)];
    g = __popcll(__ballot(lane < a.n_groups && gs <= s)) - 1;
    start = __builtin_amdgcn_readlane(gs, max(g, 0));
    next = __builtin_amdgcn_readlane(gs, g + 1);
    pre = __builtin_amdgcn_readlane(pl, max(g, 0));
  } else if (a.n_groups) {
    g = last_at_most(a.group_starts, a.n_groups, s);
    start = a.group_starts[max(g, 0)];
    next = a.group_starts[g + 1];
    pre = a.prefix_lens[max(g, 0)];
  }
  const bool in = q.row >= 0 && q.row < a.R;
  q.len = a.lens[in ? q.row : 0];
  q.ok = in && len_ok(a, q.len) && q.q0 >= 0 && end <= a.n_q;
  q.m = queries_of(q.q0, end, a.n_q);
  q.pre = 0;
  q.first = -1;
  if (g >= 0 && s < next && pre != 0) {
    q.pre = pre;
    q.first = min(max(start, 0), a.n_seqs - 1);
    q.ok = q.ok && pre > 0 && (int64_t)pre + q.m <= q.len;
  }
  return q;
}

// Whether row `row` can lend its first `pre` tokens.
__device__ __forceinline__ bool lends(const Attn& a, int row, int pre) {
  return row >= 0 && row < a.R && a.lens[row] >= pre && len_ok(a, a.lens[row]);
}

// ---------------------------------------------------------------------------
// Tiles of K and V in LDS
// ---------------------------------------------------------------------------
// A tile is kTile rows of DP halves, in 16-byte chunks; chunk c of row r lies at
// position c ^ swizzle(r), so that the 16 rows that a product's operand reads at
// one chunk fall into 16 different positions of the 256 bytes of all banks.
template <int DP>
struct Geo {
  static constexpr int NC = DP / 8;       // chunks of a row
  static constexpr int RPI = 64 / NC;     // rows that one load of a wave brings
  static constexpr int NI = kTile / RPI;  // loads of a tile
  static constexpr int BYTES = kTile * DP * 2;
};
template <int DP>
__device__ __forceinline__ int swizzle(int row) {
  return DP == 64 ? (row >> 1) & 7 : row & 15;
}

// LDS <- global, 16 bytes a lane: lane i's bytes land at lds + 16 i.  No register
// receives them, and the compiler does not count them: wait_loads<n>() waits
// until at most n of the wave's newest are on their way.  Nor does it keep the
// instructions' distances here: a load takes m0 one wait state after its write, and
// a scalar address five after a write by the vector unit (a lane read back, say).
// The copy of the address is that state, and leaves a scalar write, which needs none.
// (The compiler warns that it keeps m0 for itself; it is to know that m0 changes.)
__device__ __forceinline__ void load_lds(uint32_t lds, const char* base, uint32_t off) {
  const char* copy;
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0"
               : "=&s"(copy)
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void load_lds(uint32_t lds, const char* addr) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds), "v"(addr)
               : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// This thread's lane, as a value that the compiler does not know: what a rare path
// computes from it is not kept in registers through the loop around it.
__device__ __forceinline__ int rare_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

struct Source {           // where a workgroup's tokens come from
  const int32_t* list;    // LDS: pages of blocks block0 .. of the table row, -1 if bad
  int block0, lo, hi;     // tokens outside [lo, hi) do not exist for it
  int shift, pmask, nc;   // of the page; chunks of a head's row in use
  uint32_t page_bytes, row_bytes;
};

// Lane i (mod 32) knows token t0 + i of a tile: its page, -1 if it does not exist, and
// where its row begins in a layer's pool (of some row, if it does not exist).
struct TileAt {
  int page;
  uint32_t lo, hi;
};
__device__ __forceinline__ TileAt tile_at(const Source& s, int t0) {
  const int t = t0 + (threadIdx.x & 31);
  TileAt at;
  at.page = t >= s.lo && t < s.hi ? s.list[(t >> s.shift) - s.block0] : -1;
  const uint64_t off = (uint64_t)(uint32_t)max(at.page, 0) * s.page_bytes +
                       (uint64_t)(uint32_t)(t & s.pmask) * s.row_bytes;
  at.lo = (uint32_t)off;
  at.hi = (uint32_t)(off >> 32);
  return at;
}

// Issues loads i0 .. i0 + N - 1 of the NI of a tile of a pool (pointing at the kv
// head's channels) to the tile at LDS address lds.  Always N loads, so that
// wait_loads() can count them.  If the rows of a load lie in one page and the head
// fills the tile's width, its address is scalar but for a lane's fixed offset.
// Chunks behind the head's keep what they held.
template <int DP, int N>
__device__ __forceinline__ void load_tile(const Source& s, const char* pool, uint32_t lds, const TileAt& at,
                                          bool full, int i0 = 0) {
  using Ge = Geo<DP>;
  if (full && s.pmask >= Ge::RPI - 1 && s.nc == Ge::NC) {
    const int lane = threadIdx.x & 63, lrow = lane / Ge::NC, lc = lane % Ge::NC;
#pragma unroll
    for (int j = 0; j < N; j++) {
      const int i = i0 + j;
      const uint64_t off = (uint64_t)(uint32_t)__builtin_amdgcn_readlane(at.hi, i * Ge::RPI) << 32 |
                           (uint32_t)__builtin_amdgcn_readlane(at.lo, i * Ge::RPI);
      load_lds(lds + i * 1024, pool + off, lrow * s.row_bytes + (lc ^ swizzle<DP>(i * Ge::RPI + lrow)) * 16);
    }
  } else {
    const int lane = rare_lane(), lrow = lane / Ge::NC, lc = lane % Ge::NC;
#pragma unroll 1
    for (int i = i0; i < i0 + N; i++) {
      const int row = i * Ge::RPI + lrow, c = lc ^ swizzle<DP>(row);
      const uint64_t off = (uint64_t)(uint32_t)__shfl(at.hi, row) << 32 | (uint32_t)__shfl(at.lo, row);
      if (c < s.nc) load_lds(lds + i * 1024, pool + off + c * 16);
    }
  }
}

// Before the values of a tile of which some token does not exist or some query does
// not see some token: a value there that is no finite number must not meet the
// zero weight of such a query.  Rows of tokens that do not exist (which hold
// anything) become zeros, and so does every value that is no finite number; returns
// whether there was one: add_odd() gives it to the queries that see it.
// kBatch: chunks that are read together, as registers allow.
template <int DP, int kBatch>
__device__ __forceinline__ bool clean_values(char* tile, int pages) {
  using Ge = Geo<DP>;
  const int lane = rare_lane();
  bool odd = false;
  static_assert(Ge::NI % kBatch == 0, "");
#pragma unroll 1
  for (int i0 = 0; i0 < Ge::NI; i0 += kBatch) {
    u4* at = (u4*)(tile + i0 * 1024 + lane * 16);
    u4 x[kBatch];
    int page[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; i++) {
      x[i] = at[i * 64];
      page[i] = __shfl(pages, (i0 + i) * Ge::RPI + lane / Ge::NC);
    }
#pragma unroll
    for (int i = 0; i < kBatch; i++) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const uint32_t y = x[i][j];
        const uint32_t keep = ((y & 0x7C00u) == 0x7C00u ? 0 : 0xFFFFu) |
                              ((y & 0x7C000000u) == 0x7C000000u ? 0 : 0xFFFF0000u);
        odd |= page[i] >= 0 && keep != 0xFFFFFFFFu;
        x[i][j] = page[i] >= 0 ? y & keep : 0;
      }
      at[i * 64] = x[i];
    }
  }
  wait_lds();
  return __any(odd);
}

struct Item {
  int head, heads;          // first kv head, and how many
  int q0, rows;             // first query; rows = queries x heads of the kv head
  int lo, hi;               // tokens
  int lim0;                 // tokens that the first query sees (each later one 1 more)
  int trow;                 // table row
  int splits, split;        // of the tokens
  int slot0;                // first partial of this kind
  int row_tile, row_tiles;  // this workgroup's first row tile and its stride
  // of a sequence's rest: whether this item says where its queries' sums are, and what
  // that takes
  bool says, ok;
  int pre, first, q_end;
  int lender;               // direct: table row that the first `pre` tokens are read through
};

__device__ __forceinline__ int64_t part_at(const Attn& a, const Item& it, int head, int row) {
  return ((int64_t)(it.slot0 + it.split) * a.n_q + it.q0 + row / a.G) * a.H + head * a.G + row % a.G;
}

// The two stretches of tokens of a direct item, or an item's only one.
template <class A>
__device__ __forceinline__ int ranges_of(const A& a, const Item& it) { return a.direct && it.pre > 0 ? 2 : 1; }
__device__ __forceinline__ Item range_of(const Item& it, int ranges, int i) {
  Item r = it;
  if (ranges == 2 && i == 0) {
    r.lo = 0;
    r.hi = it.pre;
    r.trow = it.lender;
  }
  return r;
}
__device__ __forceinline__ uint16_t* out_at(const Attn& a, const Item& it, int head, int row) {
  return a.out + (it.q0 + row / a.G) * a.out_stride + (int64_t)(head * a.G + row % a.G) * a.d;
}
__device__ __forceinline__ float* lse_at(const Attn& a, const Item& it, int head, int row) {
  return a.lse + (int64_t)(it.q0 + row / a.G) * a.H + head * a.G + row % a.G;
}
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? -__builtin_inff() : (m + log2f(l)) * 0.693147180559945309f;
}
// A sum over its weights' sum, given as 1 / l, or 0 where nothing weighed anything: what
// the sum holds then (zero times what is no number, say) does not count.
__device__ __forceinline__ f4 quotient_of(f4 x, float inv) { return inv == 0.0f ? f4{0, 0, 0, 0} : x * inv; }
__device__ __forceinline__ void store_out(uint16_t* to, f4 x) {  // 4 channels
  ushort4 r;
  r.x = float_to_half_bits(x[0]);
  r.y = float_to_half_bits(x[1]);
  r.z = float_to_half_bits(x[2]);
  r.w = float_to_half_bits(x[3]);
  *(ushort4*)to = r;
}

// tokens that the query of a row sees
__device__ __forceinline__ int row_lim(const Attn& a, const Item& it, int row) {
  return min(it.hi, it.lim0 + min(row, it.rows - 1) / a.G);
}

// ---------------------------------------------------------------------------
// One wave's part: 16 RT query rows against its tiles
// ---------------------------------------------------------------------------
// Scores are computed transposed, S^T = K Q^T, so that a lane holds scores of one
// query (its column, lane & 15) for tokens 4 (lane >> 4) .. + 3 of each half tile.
// That is the layout in which O^T = V^T P^T takes P as its second operand, if
// the depth of that product runs over the tokens in the same order, which V's
// transposing reads choose freely: P never leaves its registers.
// Byte offsets of a lane's operands in a tile.  For the scores: row lane & 15, chunk
// 4 ks + lane / 16, which is at k ^ 64 ks.  For the values: the 8 bytes that its group
// of 16 lanes transposes, block b at v ^ 32 b.  Rows 16 further on have the same
// swizzle, so the second half of a tile is an immediate.
template <int DP>
struct Places {
  int k, v;
  __device__ __forceinline__ Places() {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4, row = 4 * g + (n >> 2);
    k = n * (DP * 2) + (g ^ swizzle<DP>(n)) * 16;
    v = row * (DP * 2) + (((n & 3) >> 1) ^ swizzle<DP>(row)) * 16 + (n & 1) * 8;
  }
  // the same, not to be kept for every block in registers through the loop
  __device__ __forceinline__ Places fresh() const {
    Places p = *this;
    asm volatile("" : "+v"(p.k), "+v"(p.v));
    return p;
  }
};

// One instruction, of the compiler's making: it keeps the distance to the products
// whose results these are, which it would not to a statement of assembly.
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

template <int DP, int RT>
struct Wave {
  static constexpr int KS = DP / 32, NB = DP / 16;
  h8 q[RT][KS];
  f4 o[RT][NB];
  float m[RT], l[RT];          // reference exponent (-inf: none yet), sum

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < RT; r++) {
      m[r] = -__builtin_inff();
      l[r] = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; b++) o[r][b] = f4{0, 0, 0, 0};
    }
  }

  // Queries of rows row0 .. row0 + 16 RT - 1 (row = query x heads of the kv head +
  // head); rows past the item's are zeros that see everything.
  __device__ __forceinline__ void load_queries(const Attn& a, const Item& it, int head, int row0) {
    const int n = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int r = 0; r < RT; r++) {
      const int row = row0 + r * 16 + n;
      const bool in = row < it.rows;
      const int qi = in ? row / a.G : 0, h = head * a.G + (in ? row % a.G : 0);
      const uint16_t* from = a.q + (it.q0 + qi) * a.q_stride + (int64_t)h * a.d;
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        const int ch = ks * 4 + g;
        q[r][ks] = __builtin_bit_cast(h8, in && ch < a.d / 8 ? *(const uint4*)(from + ch * 8) : uint4{0, 0, 0, 0});
      }
    }
    // negated queries stand for a negative scale, queries of 0 for a scale of 0, so
    // that the largest product has the largest score and the exponent's scale is positive
    if (a.scale <= 0) {
      const uint32_t keep = a.scale == 0 ? 0 : 0xFFFFFFFFu, flip = a.scale < 0 ? 0x80008000u : 0;
#pragma unroll
      for (int r = 0; r < RT; r++)
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
          uint4 z = __builtin_bit_cast(uint4, q[r][ks]);
          z = uint4{(z.x & keep) ^ flip, (z.y & keep) ^ flip, (z.z & keep) ^ flip, (z.w & keep) ^ flip};
          q[r][ks] = __builtin_bit_cast(h8, z);
        }
    }
  }

  // LDS operands are read in batches before the products that use them: one wait
  // for LDS instead of one per product (left to itself the compiler saves the
  // registers).  between(): called once the first batch's products are under way.
  static constexpr int KB = KS < 2 ? KS : 2, VB = NB < 4 ? NB : 4;  // of a batch
  template <class F>
  __device__ __forceinline__ void scores(const char* kt, const Places<DP>& at, f4 (&s)[RT][2], F between) {
#pragma unroll
    for (int r = 0; r < RT; r++) s[r][0] = s[r][1] = f4{0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < KS; x += KB) {
      h8 k[KB][2];
#pragma unroll
      for (int y = 0; y < KB; y++)
#pragma unroll
        for (int sub = 0; sub < 2; sub++)
          k[y][sub] = *(const h8*)(kt + (at.k ^ ((x + y) * 64)) + sub * 16 * DP * 2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int y = 0; y < KB; y++)
#pragma unroll
        for (int sub = 0; sub < 2; sub++)
#pragma unroll
          for (int r = 0; r < RT; r++)
            s[r][sub] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[y][sub], q[r][x + y], s[r][sub], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (x == 0) between();
    }
  }

  // Scores of tokens that do not exist, or that a query does not see, become -inf.
  __device__ __forceinline__ void mask(const Attn& a, const Item& it, int row0, f4 (&s)[RT][2], int t0,
                                       int pages) {
    const int lane = rare_lane(), g = lane >> 4;
    int lim[RT];
#pragma unroll
    for (int r = 0; r < RT; r++) lim[r] = row_lim(a, it, row0 + r * 16 + (lane & 15));
#pragma unroll
    for (int sub = 0; sub < 2; sub++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int tok = sub * 16 + 4 * g + i;
        const int t = __shfl(pages, tok) >= 0 ? t0 + tok : 0x7FFFFFFF;
#pragma unroll
        for (int r = 0; r < RT; r++) s[r][sub][i] = t < lim[r] ? s[r][sub][i] : -__builtin_inff();
      }
  }

  // The reference exponents of a tile's weights.  m is raised only where a score
  // passes it by kSlack, so most tiles need neither the maximum over the lanes nor a
  // rescaling of o.  peaks() finds the lane's largest scores and whether one does.
  __device__ __forceinline__ bool peaks(const f4 (&s)[RT][2], float c, float (&mx)[RT]) const {
    bool raise = false;
#pragma unroll
    for (int r = 0; r < RT; r++) {
      mx[r] = max3(max3(s[r][0][0], s[r][0][1], s[r][0][2]),
                   max3(s[r][0][3], s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3]));
      raise |= mx[r] * c > m[r] + (kSlack + kLift);
    }
    return raise;
  }
  __device__ __forceinline__ void reference(bool raise, const float (&mx)[RT], float c) {
    if (__builtin_expect(__any(raise), 0)) {
#pragma unroll
      for (int r = 0; r < RT; r++) {
        float x = mx[r];
        x = fmaxf(x, __shfl_xor(x, 16));
        x = fmaxf(x, __shfl_xor(x, 32));
        const float nm = fmaxf(m[r], x * c - kLift);
        const float f = nm == m[r] ? 1.0f : __builtin_amdgcn_exp2f(m[r] - nm);
        m[r] = nm;
        l[r] *= f;
#pragma unroll
        for (int b = 0; b < NB; b++) o[r][b] *= f;
      }
    }
  }
  // A row's sum of weights, over the lanes.  Against a reference of infinity, which a
  // score past binary32's range gives, they came out as 0: exp(inf - inf) is no number.
  __device__ __forceinline__ float sum(int r) const {
    float x = l[r];
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return m[r] == __builtin_inff() ? __builtin_nanf("") : x;
  }
  // Scores to weights, which are summed before they are rounded.
  __device__ __forceinline__ void weights(const f4 (&s)[RT][2], float c, h8 (&p)[RT]) {
#pragma unroll
    for (int r = 0; r < RT; r++) {
      float w[8];
      const float mu = m[r] == -__builtin_inff() ? 0.0f : m[r];
#pragma unroll
      for (int e = 0; e < 8; e++)
        w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][e >> 2][e & 3], c, -mu));
      l[r] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
#pragma unroll
      for (int e = 0; e < 8; e++) p[r][e] = (_Float16)w[e];  // rounded to nearest
    }
  }

  // o += V^T P^T
  template <class F>
  __device__ __forceinline__ void values(const char* vt, const Places<DP>& at, const h8 (&p)[RT], F between) {
#pragma unroll
    for (int x = 0; x < NB; x += VB) {
      h8 v[VB];
#pragma unroll
      for (int y = 0; y < VB; y++) {
        union { s4 x[2]; h8 a; } u;
#pragma unroll
        for (int sub = 0; sub < 2; sub++)
          u.x[sub] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s4*)(vt + (at.v ^ ((x + y) * 32)) + sub * 16 * DP * 2));
        v[y] = u.a;
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int y = 0; y < VB; y++)
#pragma unroll
        for (int r = 0; r < RT; r++)
          o[r][x + y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[y], p[r], o[r][x + y], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (x == 0) between();
    }
  }
};

// ---------------------------------------------------------------------------
// One workgroup: a tile of rows against a split of the tokens
// ---------------------------------------------------------------------------
// NW waves of a workgroup; TILES tiles of K and V: one for each wave, or a ring
template <int DP, int NW, int TILES>
struct Shared {
  static constexpr int kList = 512;  // table entries staged at a time
  __attribute__((aligned(1024))) char tile[TILES][2][Geo<DP>::BYTES];  // then the sums of the waves
  int32_t list[kList];
  float m[NW][32], l[NW][32], scale[NW][32];
  uint32_t odd;  // clean_values() found something
  uint32_t bad;  // a page met so far is outside the pool
};

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char*)(char*)p);
}

// What both ways of working share: the split's tiles, the pages of a stretch of them.
template <int DP, class Sh>
struct Tokens {
  static constexpr int kThreads = sizeof(Sh::m) / 128 * 64;
  Source src;
  int first, last;  // tiles
  int list_tiles;   // tiles whose pages the list holds, wherever in a page they begin
  bool bad;         // a page of this or an earlier stretch is outside the pool

  __device__ __forceinline__ bool start(const Attn& a, const Item& it, Sh& sh) {
    const Split sp = split_of(it.lo, it.hi, it.splits);
    if (it.split >= sp.used) return false;
    first = sp.tile0 + it.split * sp.per;
    last = min(first + sp.per, sp.tile0 + sp.tiles);
    const uint32_t row_bytes = (uint32_t)a.C * 2;
    src = Source{sh.list, 0, it.lo, it.hi, a.shift, a.P - 1, a.d / 8, row_bytes * (uint32_t)a.P, row_bytes};
    list_tiles = (int)((int64_t)(Sh::kList - 1) * a.P / kTile) - 1;
    return true;
  }
  // the chunks behind the head's row stay zero
  __device__ __forceinline__ void clear_tiles(const Attn& a, Sh& sh) {
    if (a.d == DP) return;
    __syncthreads();
    for (int i = threadIdx.x; i < (int)sizeof(sh.tile) / 16; i += kThreads)
      ((uint4*)sh.tile)[i] = uint4{0, 0, 0, 0};
  }
  // pages of the tokens of tiles [base, stop)
  __device__ __forceinline__ void stretch(const Attn& a, const Item& it, Sh& sh, int base,
                                          int stop) {
    const int b0 = max(base * kTile, it.lo) >> a.shift;
    const int b1 = (min(stop * kTile, it.hi) - 1) >> a.shift;
    __syncthreads();  // the list and the tiles are free
    for (int i = threadIdx.x; i <= b1 - b0; i += kThreads) {
      const int page = a.tables[(int64_t)it.trow * a.B + b0 + i];
      const bool ok = page >= 0 && page < a.N;
      sh.list[i] = ok ? page : -1;
      if (!ok) sh.bad = 1;
    }
    __syncthreads();
    bad = __builtin_amdgcn_readfirstlane(sh.bad) != 0;
    if (bad && threadIdx.x == 0) atomicOr(a.status, kBadPage);
    src.block0 = b0;
  }
  __device__ __forceinline__ bool full(int tile) const {  // every token of the tile exists
    return !bad && tile * kTile >= src.lo && (tile + 1) * kTile <= src.hi;
  }
  // tiles behind this one nobody up to row `row` sees
  __device__ __forceinline__ int seen_end(const Attn& a, const Item& it, int row) const {
    return min(last, (row_lim(a, it, row) + kTile - 1) / kTile);
  }
  // After the sums of rows [row0, row1) are stored: what clean_values() took out, for the
  // rows that see it (a sum with such a value is an infinity or no number whatever
  // the weight, and stays so where the value was counted already).  Rare, and slow.
  // empty(head, row): of a direct item, whether nothing weighed anything for a row.
  template <int kThreads, class A, class F>
  __device__ __forceinline__ void add_odd(const A& a, const Item& it, Sh& sh, int ranges, int row0, int row1, F empty) {
    const int tid = kThreads - 1 - threadIdx.x;  // nothing here is worth sharing with the loops above
    row1 = min(row1, it.rows);
#pragma unroll 1
    for (int range = 0; range < ranges; range++) {
      const Item cur = range_of(it, ranges, range);
      if (!start(a, cur, sh)) continue;
      const int end = min(seen_end(a, cur, row1 - 1) * kTile, cur.hi);
#pragma unroll 1
      for (int t = max(first * kTile, cur.lo); t < end; t++) {
        const int page = a.tables[(int64_t)cur.trow * a.B + (t >> a.shift)];
        if (page < 0 || page >= a.N) continue;
        const char* v = a.v + (uint64_t)(uint32_t)page * src.page_bytes +
                        (uint64_t)(uint32_t)(t & src.pmask) * src.row_bytes + it.head * a.d * 2;
#pragma unroll 1
        for (int i = tid; i < it.heads * a.d; i += kThreads) {
          const float x = half_bits_to_float(((const uint16_t*)v)[i]);
          if (x - x == 0.0f) continue;
          const int head = it.head + i / a.d, ch = i % a.d;
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
};

// The exponent's scale: scores are c (q . k) in units of log 2.
__device__ __forceinline__ float log2_scale(const Attn& a) {
  return a.scale == 0 ? 1.0f : fabsf(a.scale) * 1.44269504088896341f;
}

// Few rows: every wave holds all 16 RT of a row tile of its kv head.  The waves of a
// head (all, or half of them, or one, as the item has one, two or four heads) take the
// split's token tiles in turn; the waves share nothing until the end.  Each has room
// for one tile of K and one of V: the next K is on its way while the weights and the
// values are computed, the next V while the scores are.
template <int DP, int RT, int kWaves, class A>
__device__ __forceinline__ void run_split(const A& a, const Item& it, Shared<DP, kWaves, kWaves>& sh) {
  constexpr int kThreads = 64 * kWaves;
  using Ge = Geo<DP>;
  using W = Wave<DP, RT>;
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  Tokens<DP, Shared<DP, kWaves, kWaves>> tk;
  if (!a.direct && !tk.start(a, it, sh)) return;
  const int ranges = ranges_of(a, it);
  const Places<DP> at_lane;
  const int turn = kWaves / it.heads;  // waves of a head
  const int head = it.head + wave / turn;
  const char *kp = a.k + head * a.d * 2, *vp = a.v + head * a.d * 2;
  char *kt = sh.tile[wave][0], *vt = sh.tile[wave][1];
  const uint32_t klds = lds_address(kt), vlds = klds + Ge::BYTES;
  const float c = log2_scale(a);
  const int row_tiles = (it.rows + 16 * RT - 1) / (16 * RT);

  for (int rt = it.row_tile; rt < row_tiles; rt += it.row_tiles) {
    W w;
    w.clear();
    w.load_queries(a, it, head, rt * 16 * RT);
    tk.clear_tiles(a, sh);
    if (threadIdx.x == 0) sh.odd = sh.bad = 0;
#pragma unroll 1
    for (int range = 0; range < ranges; range++) {
      const Item cur = range_of(it, ranges, range);
      if (a.direct && !tk.start(a, cur, sh)) continue;
      const int min_lim = row_lim(a, cur, rt * 16 * RT);
      const int end = tk.seen_end(a, cur, (rt + 1) * 16 * RT - 1);
      for (int base = tk.first; base < end; base += tk.list_tiles) {
        const int stop = min(base + tk.list_tiles, end);
        tk.stretch(a, cur, sh, base, stop);
        // the tile in hand, where its tokens are, whether its queries see all of it; the
        // next one
        int tile = base + wave % turn, next;
        TileAt at{-1, 0, 0}, next_at{-1, 0, 0};
        bool all = false, more = false, full = false;
        auto look = [&](int nt) {
          next = nt;
          more = nt < stop;
          full = more && tk.full(nt);
          if (more) next_at = tile_at(tk.src, nt * kTile);
        };
        auto load_k = [&] { if (more) load_tile<DP, Ge::NI>(tk.src, kp, klds, next_at, full); };
        auto load_v = [&] { if (more) load_tile<DP, Ge::NI>(tk.src, vp, vlds, next_at, full); };
        auto step = [&] {
          tile = next;
          at = next_at;
          all = full && (next + 1) * kTile <= min_lim;
        };
        look(tile);
        load_k();
        load_v();
        step();
        while (tile < stop) {
          f4 s[RT][2];
          h8 p[RT];
          look(tile + turn);
          wait_loads<Ge::NI>();
          w.scores(kt, at_lane.fresh(), s, [] {});
          wait_lds();
          load_k();
          if (!all) w.mask(a, cur, rt * 16 * RT, s, tile * kTile, at.page);
          float mx[RT];
          const bool raise = w.peaks(s, c, mx);
          w.reference(raise, mx, c);
          w.weights(s, c, p);
          if (more) wait_loads<Ge::NI>(); else wait_loads<0>();
          if (!all && clean_values<DP, RT == 1 ? 4 : 1>(vt, at.page)) sh.odd = 1;
          w.values(vt, at_lane.fresh(), p, [] {});
          wait_lds();
          load_v();
          step();
        }
      }
    }
    // the waves' sums together, against the largest reference exponent
#pragma unroll
    for (int r = 0; r < RT; r++) {
      const float l = w.sum(r);
      if (g == 0) {
        sh.m[wave][r * 16 + n] = w.m[r];
        sh.l[wave][r * 16 + n] = l;
      }
    }
    __syncthreads();  // all waves are done with their tiles
    constexpr int kQuads = W::NB * 4;  // 4-channel groups of a row
    static_assert(sizeof(sh.tile) >= (size_t)kWaves * 16 * RT * kQuads * 16, "room for the sums");
    f4* sums = (f4*)sh.tile;           // [wave][row][quad], quads rotated by row
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
      for (int b = 0; b < W::NB; b++)
        sums[(wave * 16 * RT + r * 16 + n) * kQuads + ((b * 4 + g + r * 16 + n) & (kQuads - 1))] = w.o[r][b];
    if (tid < 16 * RT * it.heads) {
      const int x = tid % (16 * RT), hh = tid / (16 * RT), w0 = hh * turn;
      // All waves' are read, other heads' for nothing: without conditions, together
      // (where two row tiles take the registers, one after the other).
      constexpr int kTogether = RT == 1 ? kWaves : 1;
      float m = -__builtin_inff(), l = 0.0f;
#pragma unroll kTogether
      for (int y = 0; y < kWaves; y++) {
        const float my = sh.m[(w0 + y) % kWaves][x];
        m = y < turn ? fmaxf(m, my) : m;
      }
#pragma unroll kTogether
      for (int y = 0; y < kWaves; y++) {
        // a wave without a reference has weighed nothing, or only what is no number
        const float my = sh.m[(w0 + y) % kWaves][x], ly = sh.l[(w0 + y) % kWaves][x];
        const float f = my == m ? 1.0f : my == -__builtin_inff() && ly != 0.0f
                            ? 1.0f : __builtin_amdgcn_exp2f(my - m);
        if (y < turn) {
          sh.scale[w0 + y][x] = f;
          l += f * ly;
        }
      }
      const int row = rt * 16 * RT + x;
      if (a.direct) {
        sh.l[w0][x] = l == 0.0f ? 0.0f : 1.0f / l;
        if (row < it.rows && a.lse) *lse_at(a, it, it.head + hh, row) = lse_of(m, l);
      } else if (row < it.rows) {
        const int64_t at = part_at(a, it, it.head + hh, row);
        a.ml[2 * at] = m;
        a.ml[2 * at + 1] = l;
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < it.heads * 16 * RT * kQuads; i += kThreads) {
      const int quad = i % kQuads, row = i / kQuads % (16 * RT), hh = i / (16 * RT * kQuads), w0 = hh * turn;
      const int ch = quad * 4, gr = rt * 16 * RT + row;
      if (gr >= it.rows || ch >= a.d) continue;
      float f[kWaves];
      f4 part[kWaves], x{0, 0, 0, 0};
#pragma unroll
      for (int y = 0; y < kWaves; y++) {
        const int of = (w0 + y) % kWaves;
        f[y] = sh.scale[of][row];
        part[y] = sums[(of * 16 * RT + row) * kQuads + ((quad + row) & (kQuads - 1))];
      }
#pragma unroll
      for (int y = 0; y < kWaves; y++)
        if (y < turn) x += f[y] * part[y];
      if (a.direct) store_out(out_at(a, it, it.head + hh, gr) + ch, quotient_of(x, sh.l[w0][row]));
      else *(f4*)(a.part + part_at(a, it, it.head + hh, gr) * a.d + ch) = x;
    }
    __syncthreads();  // m, l and scale are free
    if (sh.odd)
      tk.template add_odd<kThreads>(a, it, sh, ranges, rt * 16 * RT, (rt + 1) * 16 * RT, [&](int h, int row) {
        return sh.l[(h - it.head) * turn][row - rt * 16 * RT] == 0.0f;
      });
    __syncthreads();
  }
}

// Many rows: a wave holds 16 RT of the 16 RT kWaves rows, all waves read the same token
// tiles from a ring; each loads its part of a tile, kStages - 2 tiles ahead, and one
// barrier a tile both publishes it and frees the slot that is filled next.
template <int DP, int RT, int kWaves, int kStages, class A>
__device__ __forceinline__ void run_ring(const A& a, const Item& it, Shared<DP, kWaves, kStages>& sh) {
  constexpr int kThreads = 64 * kWaves;
  using Ge = Geo<DP>;
  using W = Wave<DP, RT>;
  constexpr int kMine = Ge::NI / kWaves;  // a wave's loads of a tile of K, and of V
  static_assert(kMine >= 1 && kStages == 4, "");
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Tokens<DP, Shared<DP, kWaves, kStages>> tk;
  if (!a.direct && !tk.start(a, it, sh)) return;
  const int ranges = ranges_of(a, it);
  const Places<DP> at_lane;
  const char *kp = a.k + it.head * a.d * 2, *vp = a.v + it.head * a.d * 2;
  const uint32_t lds = lds_address(sh.tile);
  const float c = log2_scale(a);
  const int tile_rows = 16 * RT * kWaves, row_tiles = (it.rows + tile_rows - 1) / tile_rows;

  for (int rt = it.row_tile; rt < row_tiles; rt += it.row_tiles) {
    const int row0 = rt * tile_rows + wave * 16 * RT;
    W w;
    w.clear();
    w.load_queries(a, it, it.head, row0);
    tk.clear_tiles(a, sh);
    if (threadIdx.x == 0) sh.odd = sh.bad = 0;
#pragma unroll 1
    for (int range = 0; range < ranges; range++) {
      const Item cur = range_of(it, ranges, range);
      if (a.direct && !tk.start(a, cur, sh)) continue;
      const int min_lim = row_lim(a, cur, rt * tile_rows);
      const int end = tk.seen_end(a, cur, (rt + 1) * tile_rows - 1);
      for (int base = tk.first; base < end; base += tk.list_tiles) {
        const int stop = min(base + tk.list_tiles, end);
        tk.stretch(a, cur, sh, base, stop);
        char* ring = sh.tile[0][0];
        auto slot_of = [&](int tile) { return (tile - base) & (kStages - 1); };
        auto load = [&](int tile) {
          if (tile >= stop) return;
          const TileAt at = tile_at(tk.src, tile * kTile);
          const uint32_t to = lds + slot_of(tile) * (2 * Ge::BYTES);
          load_tile<DP, kMine>(tk.src, kp, to, at, tk.full(tile), wave * kMine);
          load_tile<DP, kMine>(tk.src, vp, to + Ge::BYTES, at, tk.full(tile), wave * kMine);
        };
        // Behind the barrier the tile is there for all waves, and none reads the slot of
        // the one before it any more, which takes the tile kStages - 1 ahead.
        auto publish = [&] {
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
        };
        for (int i = 0; i < kStages - 1; i++) load(base + i);

        // Tiles of which every query sees all, and the tiles loaded meanwhile too, in
        // rounds of the ring's slots: no branch but one, LDS offsets are immediates, and
        // a wave's 8 rows of a tile lie in one page, whose number is read a tile ahead.
        // (A wave that finds its way through the conditions below instead spends a quarter
        // of its time on them and on addresses: 191 us against 137 for 32 requests of 64
        // heads on 81,920 tokens, the call repeated.)
        int tile = base;
        const int seen = tk.bad || base * kTile < cur.lo ? base : min(stop, min_lim / kTile);
        if (tk.src.pmask >= 7 && tk.src.nc == Ge::NC && tile + 2 * kStages - 1 <= seen) {
          const int last_page = ((min(stop * kTile, cur.hi) - 1) >> tk.src.shift) - tk.src.block0;
          auto page_of = [&](int tl) {
            return sh.list[min(((tl * kTile + wave * 8) >> tk.src.shift) - tk.src.block0, last_page)];
          };
          const int lrow = lane / Ge::NC, lc = lane % Ge::NC;
          uint32_t at_row[kMine];
  #pragma unroll
          for (int j = 0; j < kMine; j++)
            at_row[j] = (j * Ge::RPI + lrow) * tk.src.row_bytes +
                        (lc ^ swizzle<DP>((wave * kMine + j) * Ge::RPI + lrow)) * 16;
          int page = page_of(tile + kStages - 1);
          auto step = [&](auto slot_c) {
            constexpr int kSlot = decltype(slot_c)::value;
            char* kt = ring + kSlot * 2 * Ge::BYTES;
            const uint32_t to = lds + ((kSlot + kStages - 1) & (kStages - 1)) * 2 * Ge::BYTES + wave * kMine * 1024;
            f4 s[RT][2];
            h8 p[RT];
            float mx[RT];
            wait_lds();
            wait_loads<(kStages - 2) * 2 * kMine>();
            publish();
            const int next = tile + kStages - 1;
            const uint64_t off =
                (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane(page) * tk.src.page_bytes +
                (uint64_t)((uint32_t)((next * kTile + wave * 8) & tk.src.pmask) * tk.src.row_bytes);
            // A wave's loads are spread over the step: issued at once by all waves they
            // queue for hundreds of cycles, and the waves with them.
            auto load = [&](int i) {
              if (i < kMine) load_lds(to + i * 1024, kp + off, at_row[i < kMine ? i : 0]);
              else load_lds(to + Ge::BYTES + (i - kMine) * 1024, vp + off, at_row[i < kMine ? 0 : i - kMine]);
            };
            constexpr int kQuarter = kMine >= 2 ? kMine / 2 : 1;
            auto some = [&](int from) {
  #pragma unroll
              for (int i = from * kQuarter; i < (from + 1) * kQuarter && i < 2 * kMine; i++) load(i);
            };
            w.scores(kt, at_lane.fresh(), s, [&] { some(0); });
            some(1);
            page = page_of(next + 1);
            const bool raise = w.peaks(s, c, mx);
            w.reference(raise, mx, c);
            w.weights(s, c, p);
            some(2);
            w.values(kt + Ge::BYTES, at_lane.fresh(), p, [&] { some(3); });
            tile++;
          };
          do {
            step(std::integral_constant<int, 0>());
            step(std::integral_constant<int, 1>());
            step(std::integral_constant<int, 2>());
            step(std::integral_constant<int, 3>());
          } while (tile + 2 * kStages - 1 <= seen);
        }
        for (; tile < stop; tile++) {
          char* kt = ring + slot_of(tile) * (2 * Ge::BYTES);
          char* vt = kt + Ge::BYTES;
          f4 s[RT][2];
          h8 p[RT];
          float mx[RT];
          wait_lds();
          if (tile + kStages - 1 <= stop) wait_loads<(kStages - 2) * 2 * kMine>();
          else wait_loads<0>();
          publish();
          load(tile + kStages - 1);
          w.scores(kt, at_lane.fresh(), s, [] {});
          const bool all = tk.full(tile) && (tile + 1) * kTile <= min_lim;  // the same for all waves
          if (!all) {
            const int pages = tile_at(tk.src, tile * kTile).page;
            w.mask(a, cur, row0, s, tile * kTile, pages);
            if (clean_values<DP, RT == 1 ? 4 : 1>(vt, pages)) sh.odd = 1;
          }
          const bool raise = w.peaks(s, c, mx);
          w.reference(raise, mx, c);
          w.weights(s, c, p);
          w.values(vt, at_lane.fresh(), p, [] {});
        }
      }
    }
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
        if (g == 0) sh.l[wave][r * 16 + n] = inv;
        if (g == 0 && a.lse) *lse_at(a, it, it.head, row) = lse_of(w.m[r], l);
        continue;
      }
      const int64_t at = part_at(a, it, it.head, row);
      if (g == 0) {
        a.ml[2 * at] = w.m[r];
        a.ml[2 * at + 1] = l;
      }
#pragma unroll
      for (int b = 0; b < W::NB; b++)
        if (b * 16 + g * 4 < a.d) *(f4*)(a.part + at * a.d + b * 16 + g * 4) = w.o[r][b];
    }
    __syncthreads();
    if (sh.odd)
      tk.template add_odd<kThreads>(a, it, sh, ranges, rt * tile_rows, (rt + 1) * tile_rows, [&](int, int row) {
        return sh.l[(row - rt * tile_rows) / (16 * RT)][row % (16 * RT)] == 0.0f;
      });
    __syncthreads();
  }
}

// The w-th item of the launch: first (group, split, row tile, kv head), kv heads
// fastest, for the shared prefixes, then the same per sequence for what lies behind
// them.  False: nothing to do.
template <class A>
__device__ __forceinline__ bool item_of(const A& a, int w, Item& it) {
  const int pre_items = a.pre_groups * a.pre_splits * a.pre_tiles * a.kv;
  if (w < pre_items) {
    it.head = w % a.kv;
    it.heads = 1;
    w /= a.kv;
    it.row_tile = w % a.pre_tiles;
    w /= a.pre_tiles;
    it.split = w % a.pre_splits;
    it.says = false;
    const int grp = w / a.pre_splits;
    const int s0 = a.group_starts[grp], s1 = a.group_starts[grp + 1];
    it.lo = 0;
    it.hi = a.prefix_lens[grp];
    if (s0 < 0 || s1 <= s0 || s1 > a.n_seqs || it.hi <= 0) return false;
    it.trow = row_of(a, s0);
    if (it.trow < 0 || it.trow >= a.R || !len_ok(a, a.lens[it.trow]) || a.lens[it.trow] < it.hi)
      return false;
    it.q0 = a.q_starts[s0];
    const int m = queries_of(it.q0, a.q_starts[s1], a.n_q);
    if (m == 0) return false;
    it.rows = m * a.G;
    it.lim0 = it.hi;
    it.splits = a.pre_splits;
    it.slot0 = 0;
    it.row_tiles = a.pre_tiles;
    return true;
  }
  w -= pre_items;
  it.head = w % (a.kv / a.rest_heads) * a.rest_heads;
  it.heads = a.rest_heads;
  w /= a.kv / a.rest_heads;
  it.row_tile = w % a.rest_tiles;
  w /= a.rest_tiles;
  it.split = w % a.rest_splits;
  const Seq q = sequence(a, w / a.rest_splits);
  it.says = it.head == 0 && it.split == 0 && it.row_tile == 0;
  it.ok = q.ok;
  it.pre = q.pre;
  it.first = q.first;
  it.q_end = a.q_starts[w / a.rest_splits + 1];
  it.lo = q.pre;
  it.hi = q.len;
  it.trow = q.row;
  it.q0 = q.q0;
  it.splits = a.rest_splits;
  it.slot0 = a.pre_splits;
  it.row_tiles = a.rest_tiles;
  if (a.direct && q.first >= 0) {
    it.lender = row_of(a, q.first);
    it.ok = q.ok && lends(a, it.lender, q.pre);
  }
  if (!it.ok || q.m == 0) return false;
  it.rows = q.m * a.G;
  it.lim0 = q.len - q.m + 1;
  return true;
}

// Direct: outputs of a refused sequence's queries, of the item's kv heads.
__device__ __forceinline__ void refuse(const Attn& a, const Item& it) {
  if (it.row_tile != 0) return;
  const int h0 = it.head * a.G, n = it.heads * a.G;
  for (int q = begin_of(it.q0, a.n_q); q < end_of(it.q_end, a.n_q); q++) {
    for (int i = threadIdx.x; i < n * a.d; i += blockDim.x) a.out[q * a.out_stride + h0 * a.d + i] = 0;
    for (int i = threadIdx.x; a.lse && i < n; i += blockDim.x)
      a.lse[(int64_t)q * a.H + h0 + i] = -__builtin_inff();
  }
  if (it.says && threadIdx.x == 0 && it.q0 < it.q_end) atomicOr(a.status, kRefused);
}

// For the join: where the sums of a sequence's queries are.
__device__ __forceinline__ void say_used(const Attn& a, const Item& it) {
  const bool ok = it.ok && (it.first < 0 || lends(a, row_of(a, it.first), it.pre));
  const int used = ok ? split_of(0, it.pre, a.pre_splits).used |
                            split_of(it.pre, it.hi, a.rest_splits).used << 16
                      : -1;
  for (int i = begin_of(it.q0, a.n_q) + (int)threadIdx.x; i < end_of(it.q_end, a.n_q); i += blockDim.x) a.used[i] = used;
  if (!ok && threadIdx.x == 0 && it.q0 < it.q_end) atomicOr(a.status, kRefused);
}

// How an item's workgroup holds rows: all of 16 or 32 in each of four waves, which
// deal out the tokens; or 16 or 32 in each, and the waves deal out the rows.
enum { kRows16 = 0, kRows32 = 1, kRows64 = 2, kRows128 = 3 };
__host__ __device__ constexpr int rows_of(int mode) { return 16 << mode; }
constexpr int kBlock = 256, kTiles = 4;
// workgroups on a compute unit, as LDS and registers allow
__host__ __device__ constexpr int resident(int dp) { return dp == 256 ? 1 : 2; }

template <int DP, int MODE, class A>
__device__ __forceinline__ void run_item(const A& a, const Item& it, Shared<DP, 4, kTiles>& sh) {
  if constexpr (MODE <= kRows32) run_split<DP, 1 + MODE, 4>(a, it, sh);
  else run_ring<DP, MODE == kRows128 ? 2 : 1, 4, kTiles>(a, it, sh);
}

// Items of the shared prefixes and of the rest in one launch: the former keep the
// matrix cores busy, the latter HBM.
template <int DP, int PRE, int REST, bool kDirect>
__global__ __launch_bounds__(kBlock, resident(DP)) void k_attention(Call<kDirect> a, int first, int end) {
  __shared__ Shared<DP, 4, kTiles> sh;
  for (int w = first + blockIdx.x; w < end; w += gridDim.x) {
    Item it;
    const bool go = item_of(a, w, it);
    if (go) {
      if (PRE == REST || it.slot0 == 0) run_item<DP, PRE>(a, it, sh);
      else run_item<DP, REST>(a, it, sh);
    }
    if (a.direct) {
      if (!it.ok) refuse(a, it);
    } else if (it.says) {
      say_used(a, it);
    }
  }
}

// Joins the partial sums of one query's heads.  A head takes d / 4 lanes by a.join
// parts, which add up every join-th split each: with many splits it is the number of
// loads under way that counts.
__global__ __launch_bounds__(kThreads) void k_join(Attn a) {
  __shared__ f4 sums[kThreads];
  __shared__ float ms[kThreads], ls[kThreads];
  const int qi = blockIdx.x, tid = threadIdx.x;
  const int from = a.q_starts[0], to = a.q_starts[a.n_seqs], said = a.used[qi];
  if (qi < from || qi >= to) return;  // no sequence's query
  const int pre = said < 0 ? 0 : min(said & 0xFFFF, a.pre_splits);
  const int used = said < 0 ? 0 : pre + min(said >> 16, a.rest_splits);
  const int quads = a.d / 4, unit = tid / quads, quad = tid % quads;
  const int heads = kThreads / quads / a.join;  // of a workgroup
  const int part = unit % a.join, hl = unit / a.join, h = blockIdx.y * heads + hl;
  const bool in = hl < heads && h < a.H;
  const int64_t slot_step = (int64_t)a.n_q * a.H, at0 = (int64_t)qi * a.H + h;
  auto at = [&](int x) { return at0 + slot_step * (x < pre ? x : a.pre_splits + x - pre); };
  // A sum against reference `from` is worth this much against `to`; without a reference
  // it holds nothing, or only what is no number and stays so.
  auto worth = [](float from, float to) {
    return from == to || from == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(from - to);
  };
  float m = -__builtin_inff(), l = 0.0f;
  f4 o{0, 0, 0, 0};
  if (in) {
    constexpr int kBatch = 4;  // splits whose loads are issued together
    for (int x0 = part; x0 < used; x0 += kBatch * a.join) {
      float mx[kBatch], lx[kBatch];
      f4 ox[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; i++) {
        const int64_t slot = at(min(x0 + i * a.join, used - 1));
        const float2 ml = *(const float2*)(a.ml + 2 * slot);
        mx[i] = ml.x;
        lx[i] = x0 + i * a.join < used ? ml.y : 0.0f;
        ox[i] = *(const f4*)(a.part + slot * a.d + quad * 4);
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < kBatch; i++) top = fmaxf(top, lx[i] != 0.0f ? mx[i] : top);
      const float keep = worth(m, top);
      o *= keep;
      l *= keep;
      m = top;
#pragma unroll
      for (int i = 0; i < kBatch; i++) {
        // a split in which nothing weighed anything left zeros, or what is no number: it
        // counts, unless nothing weighs anything in the others either
        if (x0 + i * a.join >= used) continue;
        const float f = worth(mx[i], m);
        o += ox[i] * f;
        l += lx[i] * f;
      }
    }
  }
  if (a.join > 1) {
    sums[tid] = o;
    ms[tid] = m;
    ls[tid] = l;
    __syncthreads();
    if (!in || part) return;
    float top = m;
    for (int x = 1; x < a.join; x++) top = fmaxf(top, ms[tid + x * quads]);
    o *= worth(m, top);
    l *= worth(m, top);
    for (int x = 1; x < a.join; x++) {
      const float f = worth(ms[tid + x * quads], top);
      o += sums[tid + x * quads] * f;
      l += ls[tid + x * quads] * f;
    }
    m = top;
  } else if (!in) {
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  store_out(a.out + qi * a.out_stride + (int64_t)h * a.d + quad * 4, quotient_of(o, inv));
  if (quad == 0 && a.lse) a.lse[(int64_t)qi * a.H + h] = lse_of(m, l);
}

// How many splits and row tiles the launch has, from the call's numbers alone.
struct Plan {
  int dp, pre_splits, rest_splits, pre_tiles, rest_tiles, pre_mode, rest_mode, pre_groups, rest_heads;
  bool direct;
  size_t words;
};

// Items first .. end - 1 of the launch's list, if there is a kernel for both kinds.
template <int DP>
bool launch(bool direct, int pre, int rest, const Attn& a, int64_t first, int64_t end, hipStream_t st) {
  if (end <= first) return true;
  const int grid = (int)std::min<int64_t>(end - first, 1 << 22);
#define GO(PRE, REST, DIRECT)                                                            \
  if (direct == DIRECT && pre == PRE && rest == REST) {                                  \
    k_attention<DP, PRE, REST, DIRECT><<<grid, kBlock, 0, st>>>({a}, (int)first, (int)end); \
    return true;                                                                         \
  }
  GO(kRows16, kRows16, false) GO(kRows64, kRows64, false) GO(kRows64, kRows16, false)
  GO(kRows16, kRows16, true) GO(kRows64, kRows64, true)
  if constexpr (DP <= 128) {
    GO(kRows32, kRows32, false) GO(kRows128, kRows128, false) GO(kRows32, kRows16, false)
    GO(kRows128, kRows16, false) GO(kRows64, kRows32, false) GO(kRows128, kRows32, false)
    GO(kRows32, kRows32, true) GO(kRows128, kRows128, true)
  }
#undef GO
  return false;
}
bool launch(int dp, bool direct, int pre, int rest, const Attn& a, int64_t first, int64_t end, hipStream_t st) {
  return dp == 64    ? launch<64>(direct, pre, rest, a, first, end, st)
         : dp == 128 ? launch<128>(direct, pre, rest, a, first, end, st)
                     : launch<256>(direct, pre, rest, a, first, end, st);
}

// The smallest that holds `rows`.  Waves of 32 rows of 256 channels would not fit
// their registers.
int mode_of(int64_t rows, int dp) {
  if (rows <= 16) return kRows16;
  if (dp == 256) return kRows64;
  return rows <= 32 ? kRows32 : rows <= 64 ? kRows64 : kRows128;
}

Plan plan_of(const cg_paged_cache& c, const cg_attention& x) {
  Plan p;
  const int kv = c.channels / x.head_dim, G = x.n_heads / kv;
  p.dp = x.head_dim <= 64 ? 64 : x.head_dim <= 128 ? 128 : 256;
  // row tiles with workgroups of their own: few enough that an item's number, over
  // all heads, sequences and splits, fits 31 bits
  auto most = [&](int64_t items) { return std::max<int64_t>(1, (1 << 22) / std::max<int64_t>(1, items)); };
  const int64_t rows = (int64_t)std::max(1, std::min(x.max_q, x.n_q)) * G;
  p.rest_mode = mode_of(rows, p.dp);
  const int rest_rows = rows_of(p.rest_mode);
  p.rest_tiles = (int)std::min(most((int64_t)x.n_seqs * kv), (rows + rest_rows - 1) / rest_rows);
  const bool shared = x.n_groups > 0 && x.max_prefix > 0;
  p.pre_groups = x.n_groups;
  // rows of an average group
  const int64_t pre_rows = std::max<int64_t>(1, x.n_groups ? (x.n_q + x.n_groups - 1) / x.n_groups : 1) * G;
  p.pre_mode = mode_of(pre_rows, p.dp);
  const int pre_tile = rows_of(p.pre_mode);
  p.pre_tiles = (int)std::min(most((int64_t)x.n_groups * kv), (pre_rows + pre_tile - 1) / pre_tile);
  // As many workgroups as are resident at once on 256 compute units (a second round
  // of a few would cost as much as the first), but no shorter splits than split_of() makes.
  auto splits = [&](int64_t items, int64_t tokens, int64_t slots, int least) {
    const int64_t room = std::max<int64_t>(1, tokens / (least * kTile));
    return (int)std::max<int64_t>(1, std::min<int64_t>({slots / std::max<int64_t>(1, items), room, 64}));
  };
  const int64_t slots = 256 * resident(p.dp);
  if (x.n_groups) {
    // the prefixes of a batch take half of the slots, and leave the others to the rest,
    // unless they are long
    const int64_t items = (int64_t)x.n_groups * kv * p.pre_tiles, tokens = shared ? x.max_prefix : 0;
    p.pre_splits = splits(items, tokens, slots, kLong);
    if (items * p.pre_splits < slots * 3 / 4) p.pre_splits = splits(items, tokens, slots / 2, kLeast);
  } else {
    p.pre_splits = 0;
  }
  p.rest_splits = splits((int64_t)std::max(1, x.n_seqs) * kv * p.rest_tiles,
                         std::max(0, x.max_len - (shared ? x.max_prefix : 0)), slots, kLeast);
  // Several heads a workgroup share its start (about 5 us of latencies) and leave fewer
  // waves to wait for the one with most tiles, as long as there are workgroups enough
  // (64 sequences of 8 kv heads and up to 600 tokens behind 9,216 shared ones: the call,
  // repeated, takes 50 us with one head, 43 with two, and 52 with four, which leaves 128
  // workgroups).
  auto heads = [&](int splits) {
    int n = 1;
    while (n < 4 && p.rest_mode <= kRows32 && kv % (2 * n) == 0 &&
           (int64_t)x.n_seqs * kv / (2 * n) * p.rest_tiles * splits >= 256)
      n *= 2;
    return n;
  };
  // Sharing saves (sequences - 1) times the prefix and costs a second kernel and its
  // start, about 5 us: not for little.
  const int64_t saved = shared ? (int64_t)x.n_seqs * x.max_prefix * c.channels * 4 : 0;
  p.direct = saved <= (int64_t)16 << 20 && x.max_prefix <= 512 &&
             splits((int64_t)std::max(1, x.n_seqs) * kv * p.rest_tiles, x.max_len, slots, kLeast) == 1;
  if (p.direct) {
    p.pre_groups = 0;
    p.pre_splits = 0;
    p.rest_splits = 1;
    p.rest_heads = heads(1);
    p.words = 4;
    return p;
  }
  p.rest_heads = heads(p.rest_splits);
  p.words = (size_t)(p.pre_splits + p.rest_splits) * x.n_q * x.n_heads * (x.head_dim + 2) + x.n_q + 4;
  return p;
}

Attn view(const cg_paged_cache& c, const cg_attention& x) {
  Attn a;
  a.C = c.channels;
  a.P = c.page_tokens;
  a.shift = __builtin_ctz((unsigned)c.page_tokens);
  a.N = c.num_pages;
  a.R = c.n_rows;
  a.B = c.max_blocks;
  const int64_t layer = (int64_t)x.layer * c.num_pages * c.page_tokens * c.channels * 2;
  a.k = (const char*)c.k_pool_dev + layer;
  a.v = (const char*)c.v_pool_dev + layer;
  a.tables = c.tables_dev;
  a.lens = c.lens_dev;
  a.status = c.status_dev;
  a.H = x.n_heads;
  a.d = x.head_dim;
  a.kv = c.channels / x.head_dim;
  a.G = x.n_heads / a.kv;
  a.scale = x.scale;
  a.n_seqs = x.n_seqs;
  a.n_q = x.n_q;
  a.n_groups = x.n_groups;
  a.rows = x.rows_dev;
  a.q_starts = x.q_starts_dev;
  a.group_starts = x.group_starts_dev;
  a.prefix_lens = x.prefix_lens_dev;
  a.q = (const uint16_t*)x.q_dev;
  a.out = (uint16_t*)x.out_dev;
  a.lse = x.lse_dev;
  a.q_stride = x.q_stride;
  a.out_stride = x.out_stride;
  return a;
}

}  // namespace
}  // namespace cg

using namespace cg;

extern "C" {

int cg_attention_workspace(const cg_paged_cache* c, const cg_attention* a, size_t* bytes) {
  if (int rc = check_attention(c, a)) return rc;
  if (!bytes) return fail(CG_E_INVAL, "bytes is NULL");
  *bytes = 4 * plan_of(*c, *a).words;
  return CG_OK;
}

int cg_attention_prefix_async(const cg_paged_cache* c, const cg_attention* a, void* workspace_dev,
                              size_t workspace_bytes, void* stream) {
  if (int rc = check_attention(c, a)) return rc;
  size_t need = 0;
  if (int rc = cg_attention_workspace(c, a, &need)) return rc;
  if (a->q_stride < (int64_t)a->n_heads * a->head_dim || a->q_stride > (int64_t)1 << 40 ||
      a->out_stride < (int64_t)a->n_heads * a->head_dim || a->out_stride > (int64_t)1 << 40 ||
      (a->q_stride | a->out_stride) % 8)
    return fail(CG_E_INVAL, "q_stride and out_stride must be multiples of 8 and at least n_heads x head_dim");
  if (a->n_seqs == 0 || a->n_q == 0) return CG_OK;
  if (!a->q_starts_dev || !a->q_dev || !a->out_dev ||
      (a->n_groups > 0 && (!a->group_starts_dev || !a->prefix_lens_dev)))
    return fail(CG_E_INVAL, "NULL pointer in the call");
  if (((uintptr_t)a->q_dev | (uintptr_t)a->out_dev | (uintptr_t)c->k_pool_dev |
       (uintptr_t)c->v_pool_dev) % 16)
    return fail(CG_E_INVAL, "pools, q and out must be 16-byte aligned");
  if (!workspace_dev || (uintptr_t)workspace_dev % 16)
    return fail(CG_E_INVAL, "workspace NULL or not 16-byte aligned");
  if (workspace_bytes < need) return fail(CG_E_CAPACITY, "workspace too small");
  DeviceGuard dg(c->device);
  if (!dg.ok) return fail(CG_E_HIP, "cannot select the cache's device");
  const Plan p = plan_of(*c, *a);
  Attn v = view(*c, *a);
  v.pre_splits = p.pre_splits;
  v.rest_splits = p.rest_splits;
  v.pre_tiles = p.pre_tiles;
  v.rest_tiles = p.rest_tiles;
  v.rest_heads = p.rest_heads;
  v.pre_groups = p.pre_groups;
  v.part = (float*)workspace_dev;
  v.ml = v.part + (size_t)(p.pre_splits + p.rest_splits) * a->n_q * a->n_heads * a->head_dim;
  v.used = (int32_t*)(v.ml + (size_t)2 * (p.pre_splits + p.rest_splits) * a->n_q * a->n_heads);
  const int64_t pre = (int64_t)p.pre_groups * p.pre_splits * p.pre_tiles * v.kv;
  const int64_t rest = (int64_t)a->n_seqs * p.rest_splits * p.rest_tiles * (v.kv / p.rest_heads);
  hipStream_t st = (hipStream_t)stream;
  const int only = pre ? p.pre_mode : p.rest_mode;
  if (!launch(p.dp, p.direct, only, p.rest_mode, v, 0, pre + rest, st)) {  // unusual pairs: one after the other
    launch(p.dp, false, p.pre_mode, p.pre_mode, v, 0, pre, st);
    launch(p.dp, false, p.rest_mode, p.rest_mode, v, pre, pre + rest, st);
  }
  if (p.direct) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? CG_OK : hip_fail(e, "attention");
  }
  const int total = p.pre_splits + p.rest_splits;
  v.join = std::min(total <= 2 ? 1 : total <= 8 ? 2 : 8, kThreads / (v.d / 4));
  const int heads = kThreads / (v.d / 4) / v.join;
  k_join<<<dim3(a->n_q, (v.H + heads - 1) / heads), kThreads, 0, st>>>(v);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? CG_OK : hip_fail(e, "attention");
}

}  // extern "C"
