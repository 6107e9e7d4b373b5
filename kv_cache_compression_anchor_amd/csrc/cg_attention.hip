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

#include "cg_attention.h"
#include "cg_hostapi.h"

namespace cg {
namespace {

// Tiles of a split of shared prefixes that take all of the chip's slots and leave the rest
// to wait for them: with fewer, half of the slots are the faster choice (14 requests of
// 64 heads, 32 of K and V, on 2,005 shared tokens: 30 us with half, 34 with all).
constexpr int kLong = 32;

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
      say_used(a, it, split_of(0, it.pre, a.pre_splits).used, split_of(it.pre, it.hi, a.rest_splits).used);
    }
  }
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
  if (int rc = check_attention_strides(a)) return rc;
  if (a->n_seqs == 0 || a->n_q == 0) return CG_OK;
  if (int rc = check_attention_memory(c, a, workspace_dev, workspace_bytes, need)) return rc;
  DeviceGuard dg(c->device);
  if (!dg.ok) return fail(CG_E_HIP, "cannot select the cache's device");
  const Plan p = plan_of(*c, *a);
  Attn v = view(*c, *a, c->channels);
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
