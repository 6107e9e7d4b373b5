// Attention over a paged cache held in 4 bits (include/cachegen.h, cg_quant_attention_async).
//
// The method is cg_attention.hip's: any split of the tokens, sums against reference
// exponents that join.  The numbers s n of the cache are binary16 numbers, and are made in
// registers on the way to the products:
//   nibbles n + 8 of a 32-bit word, two at a time, become halves 1024 + (n + 8) or
//   64 + (n + 8) by one and-or (they are the low mantissa bits of 1024, or of 64), a
//   subtraction leaves n exactly, a product with s is exact by the form of s.
#include <algorithm>

#include "cg_attention.h"
#include "cg_hostapi.h"

namespace cg {
namespace {

struct QuantAttn : Attn {
  int head_bytes, groups, scales;  // of a head: codes, scales; where the scales begin
  uint32_t row_bytes, page_bytes;
};
template <bool kDirect>
struct QuantCall : QuantAttn {
  static constexpr bool direct = kDirect;
};

// ---------------------------------------------------------------------------
// Numbers
// ---------------------------------------------------------------------------
// Nibbles 0 and 4 (kHigh: 1 and 5) of a word, less 8, as halves.
template <bool kHigh>
__device__ __forceinline__ h2 nibbles(uint32_t w) {
  const uint32_t x = kHigh ? (w & 0x00F000F0u) | 0x54005400u : (w & 0x000F000Fu) | 0x64006400u;
  const _Float16 bias = kHigh ? -72.0f : -1032.0f;
  return __builtin_bit_cast(h2, x) + h2{bias, bias};
}
// 8 channels of a word, in order, times s.
__device__ __forceinline__ h8 numbers(uint32_t w, h2 s) {
  const h2 a = nibbles<false>(w) * s, b = nibbles<true>(w) * s, c = nibbles<false>(w >> 8) * s,
           d = nibbles<true>(w >> 8) * s;
  return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ h2 both(uint16_t s) {
  const _Float16 x = __builtin_bit_cast(_Float16, s);
  return h2{x, x};
}

// What a lane holds of a tile of 32 tokens.  n = lane & 15, g = lane >> 4.
// K: of tokens n and 16 + n, channels g DP / 4 .. of the head, DP / 4 of them.
// V: of tokens 4 g + i and 16 + 4 g + i (i < 4), channels n DP / 16 .., DP / 16 of them.
template <int DP>
struct Codes {
  static constexpr int KW = DP / 32;                  // words of K a token
  static constexpr int KG = DP == 256 ? 2 : 1;        // groups that they are in
  static constexpr int VW = DP == 256 ? 2 : 1;        // words of V (DP = 64: half of one is the lane's)
  uint32_t k[2][KW], v[8][VW];
  uint16_t ks[2][KG], vs[8];
};

// Byte offsets in a token's row of what a lane holds.  What lies behind the head, where
// queries are zeros and outputs nobody's, is read from its last words instead.
template <int DP>
struct Lane {
  using Co = Codes<DP>;
  static constexpr int KP = Co::KW < 4 ? Co::KW : 4;  // words of a load of K
  int k[Co::KW / KP], ks[Co::KG], v, vs;
  __device__ __forceinline__ Lane(const QuantAttn& a, int head) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int codes = head * a.head_bytes, scales = a.scales + 2 * head * a.groups;
#pragma unroll
    for (int i = 0; i < Co::KW / KP; i++) k[i] = codes + min(g * Co::KW * 4 + i * KP * 4, a.head_bytes - KP * 4);
#pragma unroll
    for (int i = 0; i < Co::KG; i++) ks[i] = scales + 2 * min(g * (DP / 4) / 32 + i, a.groups - 1);
    v = codes + (DP == 64 ? n / 2 * 4 : min(n * Co::VW * 4, a.head_bytes - Co::VW * 4));
    if (DP == 64) v = min(v, codes + a.head_bytes - 4);
    vs = scales + 2 * min(n * (DP / 16) / 32, a.groups - 1);
  }
};

// The pages of a stretch of tokens [lo, hi) of a table row, staged in LDS.
struct Pages {
  const int32_t* list;  // pages of blocks block0 .., -1 outside the pool
  int block0, lo, hi, shift, pmask;
};

// Where tile t0's tokens are.  Lane i (mod 32) knows token t0 + i: its page (of the nearest
// token there is, if it does not exist); alive: bits of the tokens that exist.
struct At {
  int page;
  uint32_t alive;
};
__device__ __forceinline__ At find(const Pages& p, int t0) {
  const int t = t0 + (threadIdx.x & 31), c = min(max(t, p.lo), p.hi - 1);
  const int page = p.list[(c >> p.shift) - p.block0];
  return {max(page, 0), (uint32_t)__ballot(t == c && page >= 0)};
}

template <int DP>
__device__ __forceinline__ void load_codes(const QuantAttn& a, const Pages& p, const Lane<DP>& ln, const At& at, int t0,
                                           Codes<DP>& x) {
  using Co = Codes<DP>;
  using KPiece = uint32_t __attribute__((ext_vector_type(Lane<DP>::KP)));
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  auto token = [&](const char* kt, const char* vt, int i, bool k) {  // pointers to a token's rows
    if (k) {
#pragma unroll
      for (int j = 0; j < Co::KW / Lane<DP>::KP; j++) {
        const KPiece y = *(const KPiece*)(kt + ln.k[j]);
#pragma unroll
        for (int e = 0; e < Lane<DP>::KP; e++) x.k[i][j * Lane<DP>::KP + e] = y[e];
      }
#pragma unroll
      for (int j = 0; j < Co::KG; j++) x.ks[i][j] = *(const uint16_t*)(kt + ln.ks[j]);
    } else {
      if constexpr (Co::VW == 2) {
        const uint2 y = *(const uint2*)(vt + ln.v);
        x.v[i][0] = y.x;
        x.v[i][1] = y.y;
      } else {
        x.v[i][0] = *(const uint32_t*)(vt + ln.v);
      }
      x.vs[i] = *(const uint16_t*)(vt + ln.vs);
    }
  };
  if (p.pmask >= 15) {  // 16 tokens lie in one page: its address is scalar
#pragma unroll
    for (int sub = 0; sub < 2; sub++) {
      const uint64_t off = (uint64_t)(uint32_t)__builtin_amdgcn_readlane(at.page, 16 * sub) * a.page_bytes +
                           (uint64_t)(uint32_t)((t0 + 16 * sub) & p.pmask) * a.row_bytes;
      const char *kb = a.k + off, *vb = a.v + off;
      token(kb + n * a.row_bytes, nullptr, sub, true);
#pragma unroll
      for (int i = 0; i < 4; i++) token(nullptr, vb + (4 * g + i) * a.row_bytes, 4 * sub + i, false);
    }
  } else {
    auto row = [&](int tok) {
      return (uint64_t)(uint32_t)__shfl(at.page, tok) * a.page_bytes +
             (uint64_t)(uint32_t)((t0 + tok) & p.pmask) * a.row_bytes;
    };
#pragma unroll
    for (int sub = 0; sub < 2; sub++) {
      token(a.k + row(16 * sub + n), nullptr, sub, true);
#pragma unroll
      for (int i = 0; i < 4; i++) token(nullptr, a.v + row(16 * sub + 4 * g + i), 4 * sub + i, false);
    }
  }
}

// Scores of a tile: S^T = K Q^T.
template <int DP, int RT>
__device__ __forceinline__ void scores(const Wave<DP, RT>& w, const Codes<DP>& x, f4 (&s)[RT][2]) {
#pragma unroll
  for (int r = 0; r < RT; r++) s[r][0] = s[r][1] = f4{0, 0, 0, 0};
#pragma unroll
  for (int sub = 0; sub < 2; sub++)
#pragma unroll
    for (int ks = 0; ks < DP / 32; ks++) {
      const h8 k = numbers(x.k[sub][ks], both(x.ks[sub][DP == 256 ? ks / 4 : 0]));
#pragma unroll
      for (int r = 0; r < RT; r++) s[r][sub] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, w.q[r][ks], s[r][sub], 0, 0, 0);
    }
}

// o += V^T P^T.  Row n of block b of V^T is channel n DP / 16 + b, so that a lane's
// channels are neighbours in its word; its tokens come together two at a time.
// kClean: some query does not see some token; numbers that are not finite become zeros and
// tokens that do not exist too.  Returns whether there was such a number.
template <int DP, int RT, bool kClean>
__device__ __forceinline__ bool values(Wave<DP, RT>& w, const Codes<DP>& x, const h8 (&p)[RT], uint32_t alive) {
  constexpr int NB = DP / 16;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  union { uint32_t u[4]; h8 h; } v[NB];
  bool odd = false;
#pragma unroll
  for (int j = 0; j < 4; j++) {  // tokens 4 g + 2 j, + 1 (j < 2), 16 + 4 g + 2 (j - 2), + 1
    const int tok = (j >> 1) * 16 + 4 * g + (j & 1) * 2;
    h2 s{__builtin_bit_cast(_Float16, x.vs[2 * j]), __builtin_bit_cast(_Float16, x.vs[2 * j + 1])};
    uint32_t there = 0xFFFFFFFFu;
    if (kClean) there = ((alive >> tok) & 1 ? 0xFFFFu : 0) | ((alive >> tok) & 2 ? 0xFFFF0000u : 0);
#pragma unroll
    for (int y = 0; y < Codes<DP>::VW; y++) {
      uint32_t w0 = x.v[2 * j][y], w1 = x.v[2 * j + 1][y];
      if (DP == 64) {
        w0 >>= 8 * (n & 1);
        w1 >>= 8 * (n & 1);
      }
      const uint32_t lo = __builtin_amdgcn_perm(w1, w0, 0x05040100u), hi = __builtin_amdgcn_perm(w1, w0, 0x07060302u);
      auto put = [&](int b, h2 z) {
        uint32_t u = __builtin_bit_cast(uint32_t, z * s);
        if (kClean) {
          const uint32_t keep = ((u & 0x7C00u) == 0x7C00u ? 0 : 0xFFFFu) | ((u & 0x7C000000u) == 0x7C000000u ? 0 : 0xFFFF0000u);
          odd |= (~keep & there) != 0;
          u &= keep & there;
        }
        v[y * 8 + b].u[j] = u;
      };
      put(0, nibbles<false>(lo));
      put(1, nibbles<false>(hi));
      put(2, nibbles<true>(lo));
      put(3, nibbles<true>(hi));
      if constexpr (DP > 64) {
        put(4, nibbles<false>(lo >> 8));
        put(5, nibbles<false>(hi >> 8));
        put(6, nibbles<true>(lo >> 8));
        put(7, nibbles<true>(hi >> 8));
      }
    }
  }
#pragma unroll
  for (int b = 0; b < NB; b++)
#pragma unroll
    for (int r = 0; r < RT; r++) w.o[r][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[b].h, p[r], w.o[r][b], 0, 0, 0);
  return kClean && __any(odd);
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
template <int DP, int RT>
struct QuantShared {
  static constexpr int kWaves = kBlock / 64;
  f4 sums[kWaves * 16 * RT * DP / 4];
  int32_t list[kList];
  float m[kWaves][16 * RT], l[kWaves][16 * RT], scale[kWaves][16 * RT];
  uint32_t odd;  // values() found something
  uint32_t bad;  // a page met so far is outside the pool
};

// Half of channel ch of kv head `head` in the row at p.
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
template <class A, class F>
__device__ __forceinline__ void add_odd(const A& a, const Item& it, int ranges, int row0, int row1, F empty) {
  const int tid = kBlock - 1 - threadIdx.x;
  row1 = min(row1, it.rows);
#pragma unroll 1
  for (int range = 0; range < ranges; range++) {
    const Item cur = range_of(it, ranges, range);
    const Split sp = split_of(cur.lo, cur.hi, cur.splits);
    if (cur.split >= sp.used) continue;
    const int first = sp.tile0 + cur.split * sp.per, last = min(first + sp.per, sp.tile0 + sp.tiles);
    const int end = min(min(last * kTile, cur.hi), row_lim(a, cur, row1 - 1));
#pragma unroll 1
    for (int t = max(first * kTile, cur.lo); t < end; t++) {
      const int page = a.tables[(int64_t)cur.trow * a.B + (t >> a.shift)];
      if (page < 0 || page >= a.N) continue;
      const char* v = a.v + (uint64_t)(uint32_t)page * a.page_bytes + (uint64_t)(uint32_t)(t & (a.P - 1)) * a.row_bytes;
#pragma unroll 1
      for (int i = tid; i < it.heads * a.d; i += kBlock) {
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

// Every wave holds all 16 RT of a row tile of its kv head.  The waves of a head (all, or
// half of them, or one, as the item has one, two or four heads) take the split's token
// tiles in turn and share nothing until the end; a wave's next tile is on its way to
// registers while it computes one.
template <int DP, int RT, class A>
__device__ __forceinline__ void run_few(const A& a, const Item& it, QuantShared<DP, RT>& sh) {
  constexpr int kWaves = kBlock / 64;
  using W = Wave<DP, RT>;
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ranges = ranges_of(a, it);
  const int turn = kWaves / it.heads;  // waves of a head
  const int head = it.head + wave / turn;
  const float c = log2_scale(a);
  const int row_tiles = (it.rows + 16 * RT - 1) / (16 * RT);
  const int list_tiles = (int)((int64_t)(kList - 1) * a.P / kTile) - 1;
  {
    const Split sp = split_of(it.lo, it.hi, it.splits);
    if (!a.direct && it.split >= sp.used) return;
  }
  const Lane<DP> ln(a, head);

  for (int rt = it.row_tile; rt < row_tiles; rt += it.row_tiles) {
    W w;
    w.clear();
    w.template load_queries<true>(a, it, head, rt * 16 * RT);
    if (tid == 0) sh.odd = sh.bad = 0;
#pragma unroll 1
    for (int range = 0; range < ranges; range++) {
      const Item cur = range_of(it, ranges, range);
      const Split sp = split_of(cur.lo, cur.hi, cur.splits);
      if (cur.split >= sp.used) continue;
      const int first = sp.tile0 + cur.split * sp.per, last = min(first + sp.per, sp.tile0 + sp.tiles);
      const int min_lim = row_lim(a, cur, rt * 16 * RT);
      // tiles behind this one nobody of these rows sees
      const int end = min(last, (row_lim(a, cur, (rt + 1) * 16 * RT - 1) + kTile - 1) / kTile);
      for (int base = first; base < end; base += list_tiles) {
        const int stop = min(base + list_tiles, end);
        const int b0 = max(base * kTile, cur.lo) >> a.shift, b1 = (min(stop * kTile, cur.hi) - 1) >> a.shift;
        __syncthreads();  // the list is free
        for (int i = tid; i <= b1 - b0; i += kBlock) {
          const int page = a.tables[(int64_t)cur.trow * a.B + b0 + i];
          const bool ok = page >= 0 && page < a.N;
          sh.list[i] = ok ? page : -1;
          if (!ok) sh.bad = 1;
        }
        __syncthreads();
        // tokens that exist for this stretch lie in its blocks
        const Pages pages{sh.list, b0, max(base * kTile, cur.lo), min(stop * kTile, cur.hi), a.shift, a.P - 1};
        auto step = [&](const Codes<DP>& x, uint32_t alive, int tile) {
          f4 s[RT][2];
          h8 p[RT];
          float mx[RT];
          scores(w, x, s);
          const bool all = alive == 0xFFFFFFFFu && (tile + 1) * kTile <= min_lim;
          if (!all) mask_scores<DP, RT>(a, cur, rt * 16 * RT, s, tile * kTile, alive);
          const bool raise = w.peaks(s, c, mx);
          w.reference(raise, mx, c);
          w.weights(s, c, p);
          if (all) values<DP, RT, false>(w, x, p, alive);
          else if (values<DP, RT, true>(w, x, p, alive)) sh.odd = 1;
        };
        Codes<DP> x0, x1;
        At at0{0, 0}, at1{0, 0};
        int tile = base + wave % turn;
        if (tile < stop) {
          at0 = find(pages, tile * kTile);
          load_codes<DP>(a, pages, ln, at0, tile * kTile, x0);
        }
        while (tile < stop) {
          const int next = tile + turn, after = next + turn;
          if (next < stop) {
            at1 = find(pages, next * kTile);
            load_codes<DP>(a, pages, ln, at1, next * kTile, x1);
          }
          step(x0, at0.alive, tile);
          if (next >= stop) break;
          if (after < stop) {
            at0 = find(pages, after * kTile);
            load_codes<DP>(a, pages, ln, at0, after * kTile, x0);
          }
          step(x1, at1.alive, next);
          tile = after;
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
    constexpr int kQuads = DP / 4;  // 4-channel groups of a row, which the lanes hold a channel of each of 4 blocks
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int b = 0; b < W::NB; b += 4) {
          const int quad = (4 * g + i) * (W::NB / 4) + b / 4, row = r * 16 + n;
          sh.sums[(wave * 16 * RT + row) * kQuads + ((quad + row) & (kQuads - 1))] =
              f4{w.o[r][b][i], w.o[r][b + 1][i], w.o[r][b + 2][i], w.o[r][b + 3][i]};
        }
    __syncthreads();
    if (sh.bad && tid == 0) atomicOr(a.status, kBadPage);
    if (tid < 16 * RT * it.heads) {
      const int x = tid % (16 * RT), hh = tid / (16 * RT), w0 = hh * turn;
      float m = -__builtin_inff(), l = 0.0f;
#pragma unroll
      for (int y = 0; y < kWaves; y++) {
        const float my = sh.m[(w0 + y) % kWaves][x];
        m = y < turn ? fmaxf(m, my) : m;
      }
#pragma unroll
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
        sh.m[w0][x] = l == 0.0f ? 0.0f : 1.0f / l;
        if (row < it.rows && a.lse) *lse_at(a, it, it.head + hh, row) = lse_of(m, l);
      } else if (row < it.rows) {
        const int64_t at = part_at(a, it, it.head + hh, row);
        a.ml[2 * at] = m;
        a.ml[2 * at + 1] = l;
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < it.heads * 16 * RT * kQuads; i += kBlock) {
      const int quad = i % kQuads, row = i / kQuads % (16 * RT), hh = i / (16 * RT * kQuads), w0 = hh * turn;
      const int ch = quad * 4, gr = rt * 16 * RT + row;
      if (gr >= it.rows || ch >= a.d) continue;
      f4 x{0, 0, 0, 0};
#pragma unroll
      for (int y = 0; y < kWaves; y++) {
        const int of = (w0 + y) % kWaves;
        const float f = sh.scale[of][row];
        const f4 part = sh.sums[(of * 16 * RT + row) * kQuads + ((quad + row) & (kQuads - 1))];
        if (y < turn) x += f * part;
      }
      if (a.direct) store_out(out_at(a, it, it.head + hh, gr) + ch, quotient_of(x, sh.m[w0][row]));
      else *(f4*)(a.part + part_at(a, it, it.head + hh, gr) * a.d + ch) = x;
    }
    __syncthreads();
    if (sh.odd)
      add_odd(a, it, ranges, rt * 16 * RT, (rt + 1) * 16 * RT,
              [&](int h, int row) { return sh.m[(h - it.head) * turn][row - rt * 16 * RT] == 0.0f; });
    __syncthreads();  // m, l, scale and the sums are free
  }
}

template <int DP, int RT, bool kDirect>
__global__ __launch_bounds__(kBlock, 2) void k_quant_attention(QuantCall<kDirect> a, int first, int end) {
  __shared__ QuantShared<DP, RT> sh;
  for (int w = first + blockIdx.x; w < end; w += gridDim.x) {
    Item it;
    if (item_of(a, w, it)) run_few<DP, RT>(a, it, sh);
    if (a.direct) {
      if (!it.ok) refuse(a, it);
    } else if (it.says) {
      say_used(a, it);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// How many splits and row tiles the launch has, from the call's numbers alone.
struct Plan {
  int dp, pre_splits, rest_splits, pre_tiles, rest_tiles, pre_mode, rest_mode, pre_groups, rest_heads;
  bool direct;
  size_t words;
};

template <int DP>
void launch(bool direct, int mode, const QuantAttn& a, int64_t first, int64_t end, hipStream_t st) {
  if (end <= first) return;
  const int grid = (int)std::min<int64_t>(end - first, 1 << 22);
#define GO(MODE, DIRECT)                                                                             \
  if (direct == DIRECT && mode == MODE)                                                              \
    k_quant_attention<DP, 1 + MODE, DIRECT><<<grid, kBlock, 0, st>>>({a}, (int)first, (int)end);
  GO(kRows16, false) GO(kRows16, true)
  if constexpr (DP <= 128) { GO(kRows32, false) GO(kRows32, true) }
#undef GO
}
void launch(int dp, bool direct, int mode, const QuantAttn& a, int64_t first, int64_t end, hipStream_t st) {
  if (dp == 64) launch<64>(direct, mode, a, first, end, st);
  else if (dp == 128) launch<128>(direct, mode, a, first, end, st);
  else launch<256>(direct, mode, a, first, end, st);
}

int mode_of(int64_t rows, int dp) { return rows <= 16 || dp == 256 ? kRows16 : kRows32; }

Plan plan_of(const cg_paged_cache& c, const cg_quant_form& f, const cg_attention& x) {
  Plan p;
  const int kv = f.channels / x.head_dim, G = x.n_heads / kv;
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
  auto splits = [&](int64_t items, int64_t tokens, int64_t slots) {
    const int64_t room = std::max<int64_t>(1, tokens / (kLeast * kTile));
    return (int)std::max<int64_t>(1, std::min<int64_t>({slots / std::max<int64_t>(1, items), room, 64}));
  };
  const int64_t slots = 512;
  p.pre_splits = x.n_groups ? splits((int64_t)x.n_groups * kv * p.pre_tiles, shared ? x.max_prefix : 0, slots) : 0;
  p.rest_splits = splits((int64_t)std::max(1, x.n_seqs) * kv * p.rest_tiles,
                         std::max(0, x.max_len - (shared ? x.max_prefix : 0)), slots);
  auto heads = [&](int splits) {
    int n = 1;
    while (n < 4 && kv % (2 * n) == 0 && (int64_t)x.n_seqs * kv / (2 * n) * p.rest_tiles * splits >= 256) n *= 2;
    return n;
  };
  // Sharing saves (sequences - 1) times the prefix and costs a second kernel and its
  // start, about 5 us: not for little.
  const int64_t saved = shared ? (int64_t)x.n_seqs * x.max_prefix * c.channels * 4 : 0;
  p.direct = saved <= (int64_t)16 << 20 && x.max_prefix <= 512 &&
             splits((int64_t)std::max(1, x.n_seqs) * kv * p.rest_tiles, x.max_len, slots) == 1;
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
              (uint32_t)r.row * (uint32_t)c->page_tokens};
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
  const int64_t pre = (int64_t)p.pre_groups * p.pre_splits * p.pre_tiles * v.kv;
  const int64_t rest = (int64_t)a->n_seqs * p.rest_splits * p.rest_tiles * (v.kv / p.rest_heads);
  hipStream_t st = (hipStream_t)stream;
  if (p.pre_mode == p.rest_mode || !pre) {
    launch(p.dp, p.direct, p.rest_mode, v, 0, pre + rest, st);
  } else {
    launch(p.dp, false, p.pre_mode, v, 0, pre, st);
    launch(p.dp, false, p.rest_mode, v, pre, pre + rest, st);
  }
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
