// What attention over paged caches shares whatever form their rows have: a call as the
// kernels see it, its items and sequences, one wave's scores, weights and sums, and the
// join of split tokens.  cg_attention.hip describes the method.
#pragma once

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
  int rest_heads;  // kv heads of a workgroup that deals out the rest's tokens: 1, 2 or 4; over 4 bits up to 8
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

// This thread's lane, as a value that the compiler does not know: what a rare path
// computes from it is not kept in registers through the loop around it.
__device__ __forceinline__ int rare_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
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
  // head); rows past the item's are zeros that see everything.  A product's depth takes the
  // channels in any order that K has too: product ks takes chunk 4 ks + lane / 16 from a
  // lane, or (kSpans) a lane's chunks are neighbours.
  template <bool kSpans = false>
  __device__ __forceinline__ void load_queries(const Attn& a, const Item& it, int head, int row0, int lane = threadIdx.x & 63) {
    const int n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int r = 0; r < RT; r++) {
      const int row = row0 + r * 16 + n;
      const bool in = row < it.rows;
      const int qi = in ? row / a.G : 0, h = head * a.G + (in ? row % a.G : 0);
      const uint16_t* from = a.q + (it.q0 + qi) * a.q_stride + (int64_t)h * a.d;
#pragma unroll
      for (int ks = 0; ks < KS; ks++) {
        const int ch = kSpans ? g * KS + ks : ks * 4 + g;
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
  // What that rounding took from each.
  __device__ __forceinline__ void rests(const f4 (&s)[RT][2], float c, const h8 (&p)[RT], h8 (&rest)[RT]) {
#pragma unroll
    for (int r = 0; r < RT; r++) {
      const float mu = m[r] == -__builtin_inff() ? 0.0f : m[r];
#pragma unroll
      for (int e = 0; e < 8; e++)
        rest[r][e] = (_Float16)(__builtin_amdgcn_exp2f(__builtin_fmaf(s[r][e >> 2][e & 3], c, -mu)) - (float)p[r][e]);
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

// The exponent's scale: scores are c (q . k) in units of log 2.
__device__ __forceinline__ float log2_scale(const Attn& a) {
  return a.scale == 0 ? 1.0f : fabsf(a.scale) * 1.44269504088896341f;
}

// kv heads of an item of a shared prefix.
__device__ __forceinline__ constexpr int prefix_heads(const Attn&) { return 1; }

// Sequence s's own tokens (direct: all of them) for the item's row tile, kv heads and split.
template <class A>
__device__ __forceinline__ bool rest_item(const A& a, int s, Item& it) {
  const Seq q = sequence(a, s);
  it.says = it.head == 0 && it.split == 0 && it.row_tile == 0;
  it.ok = q.ok;
  it.pre = q.pre;
  it.first = q.first;
  it.q_end = a.q_starts[s + 1];
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

// The w-th item of the launch: first (group, split, row tile, kv head), kv heads
// fastest, for the shared prefixes, then the same per sequence for what lies behind
// them.  False: nothing to do.
template <class A>
__device__ __forceinline__ bool item_of(const A& a, int w, Item& it) {
  const int pre_items = a.pre_groups * a.pre_splits * a.pre_tiles * (a.kv / prefix_heads(a));
  if (w < pre_items) {
    const int heads = prefix_heads(a), columns = a.kv / heads;
    it.head = w % columns * heads;
    it.heads = heads;
    w /= columns;
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
  return rest_item(a, w / a.rest_splits, it);
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

// For the join: where the sums of a sequence's queries are, in `pre` splits of its prefix and
// `rest` of its own tokens.
__device__ __forceinline__ void say_used(const Attn& a, const Item& it, int pre, int rest) {
  const bool ok = it.ok && (it.first < 0 || lends(a, row_of(a, it.first), it.pre));
  const int used = ok ? pre | rest << 16 : -1;
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

// The call on a cache whose rows stand for `channels` channels; k and v are the layer's
// pools, and the launch is the caller's to fill in.
inline Attn view(const cg_paged_cache& c, const cg_attention& x, int channels) {
  Attn a;
  a.C = channels;
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
  a.kv = channels / x.head_dim;
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
