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
  int pre_least, rest_least;  // tiles of a split, at least
};
__device__ __forceinline__ Split prefix_split(const QuantAttn& a, int hi) {
  return split_of(0, hi, a.pre_splits, a.pre_least);
}
__device__ __forceinline__ Split rest_split(const QuantAttn& a, int lo, int hi) {
  return split_of(lo, hi, a.rest_splits, a.rest_least);
}
template <bool kDirect>
struct QuantCall : QuantAttn {
  static constexpr bool direct = kDirect;
};
// The tiles of an item's tokens (of one of a direct item's stretches), and its part of them.
template <class A>
__device__ __forceinline__ Split split_of(const A& a, const Item& it) {
  return !a.direct && it.slot0 == 0 && a.pre_splits > 0 ? prefix_split(a, it.hi) : rest_split(a, it.lo, it.hi);
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
// Tiles of codes and scales in LDS
// ---------------------------------------------------------------------------
// A wave's tile is 32 tokens' rows of K and of V of one head, as they are in memory, brought
// by loads that no register receives.  n = lane & 15, g = lane >> 4.
//   K: row r of DP / 2 bytes in 16-byte chunks, chunk c at position c ^ twist(r): a lane reads
//      channels g DP / 4 .. of tokens n and 16 + n, 16 rows of one chunk each fall into 16
//      different positions of the 256 bytes of all banks.
//   V: row r = 4 g + i of a half tile at 4 i + g: a lane reads its channels of tokens
//      4 g + i, for one i four neighbouring rows.
//   scales: of each half tile, 16 tokens of K and 16 of V, a window of 8 (DP = 256: 16) bytes
//      that holds the head's, from the second half on where they begin in the middle of a
//      word; for DP = 64 one word twice.
// A lane's channels of V follow from how scales are read: a transposing read gives lane n
// those of 4 tokens at place n % 4 (DP = 64: n % 2, DP = 256: n % 8) of the window.
template <int DP>
struct Stage {
  static constexpr int ROW = DP / 2, CH = ROW / 16;    // bytes and chunks of a row
  static constexpr int RPL = 64 / CH;                  // rows of a load
  static constexpr int WIN = DP == 256 ? 16 : 8;       // bytes of a window
  static constexpr int CODES = 32 * ROW, SCALES = 16 * WIN;
  static constexpr int BYTES = 2 * CODES + 4 * SCALES;
  static constexpr int LOADS = 2 * (32 / RPL) + (DP == 256 ? 4 : 2);
  __device__ __forceinline__ static int twist(int r) { return CH == 2 ? (r >> 3) & 1 : CH == 4 ? (r >> 2) & 3 : (r >> 1) & 7; }
};

// LDS <- global, 16 or 4 bytes a lane, lane i's at lds + 16 i or 4 i.  The compiler does not
// count these loads (wait_loads does) and keeps no distances here: a load takes m0 one wait
// state after its write, and a scalar address five after a write by the vector unit; the copy
// of the address is that state, and leaves a scalar write, which needs none.
__device__ __forceinline__ void load_lds16(uint32_t lds, const char* base, uint32_t off) {
  const char* copy;
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0"
               : "=&s"(copy)
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void load_lds16(uint32_t lds, const char* addr) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(lds), "v"(addr) : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(uint32_t lds, const char* addr) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" : : "s"(lds), "v"(addr) : "memory", "m0");
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

// A lane's part in bringing tiles of one head, and in reading them.
template <int DP>
struct Head {
  using St = Stage<DP>;
  static constexpr int KPH = 16 / St::RPL ? 16 / St::RPL : 1;  // loads of a half tile
  const char *k, *v;         // the layer's pools
  uint32_t koff[KPH], voff;  // of the lane's chunk in a half tile whose rows follow one another
  const char* sbase;         // pool of the lane's scales, at their place in a row
  uint32_t soff;             // (for V: DP = 256)
  int kread, kscale, kstep, vread, vscale;
  uint32_t bytes;            // DP = 64: where the lane's channels of V are in their word
  int channel;               // the lane's first channel of V, DP / 16 of them; d or more: none

  __device__ __forceinline__ Head(const QuantAttn& a, int head) : k(a.k), v(a.v) {
    const int lane = rare_lane(), n = lane & 15, g = lane >> 4;
    const int codes = head * a.head_bytes, last = a.head_bytes / 16 - 1;
    const int row = lane / St::CH, c = lane % St::CH;
#pragma unroll
    for (int j = 0; j < KPH; j++) {
      const int r = j * St::RPL + row;
      koff[j] = (DP == 64 ? row & 15 : r) * a.row_bytes + codes + min(c ^ St::twist(r & 15), last) * 16;
    }
    const int half = row & 15;
    voff = (4 * (half & 3) + (half >> 2)) * a.row_bytes + codes + min(c, last) * 16;
    // scales
    const int odd = (head * a.groups) & 1, window = a.scales + 2 * (head * a.groups - odd);
    const int token = DP == 256 ? lane >> 2 : (lane & 31) >> 1, word = DP == 256 ? lane & 3 : DP == 64 ? 0 : lane & 1;
    soff = min(window + 4 * word, (int)a.row_bytes - 4) + token * a.row_bytes;
    sbase = DP == 256 || lane < 32 ? a.k : a.v;
    kread = DP == 64 ? n * 32 + ((g >> 1) ^ St::twist(n)) * 16 + (g & 1) * 8
                     : n * St::ROW + ((DP == 256 ? 2 * g : g) ^ St::twist(n)) * 16;
    const int kg = DP == 64 ? g >> 1 : DP == 128 ? g : 2 * g;
    kscale = n * St::WIN + 2 * (odd + min(kg, a.groups - 1));
    kstep = kg + 1 < a.groups ? 2 : 0;
    const int place = DP == 64 ? n & 1 : DP == 128 ? n & 3 : (n >> 2 & 1) * 4 + (n & 3);
    const int j = DP == 64 ? n >> 1 : DP == 128 ? n >> 2 : n >> 3;  // of the lanes of a group
    const int group = place - odd;
    const bool in = group >= 0 && group < a.groups;
    const int first = (in ? group * 32 : 0) + j * (DP / 16);
    channel = in ? first : 256;
    vread = g * St::ROW + first / 8 * 4;
    bytes = 0x0C040C00u + (first & 4 ? 0x00010001u : 0);
    vscale = (4 * g + (n >> 2)) * St::WIN + (DP == 256 ? (n & 1) * 8 : 0);
  }

  // Issues the loads of tile t0 to the stage at LDS address `lds`; always St::LOADS of them.
  __device__ __forceinline__ void load(const QuantAttn& a, const Pages& p, const At& at, int t0, uint32_t lds) const {
    const uint32_t klds = lds, vlds = lds + St::CODES, slds = lds + 2 * St::CODES;
    if (p.pmask >= 15) {  // the 16 tokens of a half tile lie in one page
      uint64_t off[2];
#pragma unroll
      for (int h = 0; h < 2; h++)
        off[h] = (uint64_t)(uint32_t)__builtin_amdgcn_readlane(at.page, 16 * h) * a.page_bytes +
                 (uint64_t)(uint32_t)((t0 + 16 * h) & p.pmask) * a.row_bytes;
      if constexpr (DP == 64) {  // a load brings both halves
        const uint64_t my = (threadIdx.x & 32) ? off[1] : off[0];
        load_lds16(klds, k + my + koff[0]);
        load_lds16(vlds, v + my + voff);
      } else {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int j = 0; j < KPH; j++) {
            load_lds16(klds + (h * KPH + j) * 1024, k + off[h], koff[j]);
            load_lds16(vlds + (h * KPH + j) * 1024, v + off[h] + 2 * j * a.row_bytes, voff);
          }
      }
#pragma unroll
      for (int h = 0; h < 2; h++) {
        load_lds4(slds + h * 2 * St::SCALES, sbase + off[h] + soff);
        if constexpr (DP == 256) load_lds4(slds + h * 2 * St::SCALES + St::SCALES, v + off[h] + soff);
      }
    } else {
      const int lane = rare_lane();
      auto row = [&](int tok) {  // where the token's row is, less that of its place in a half tile
        return (uint64_t)(uint32_t)__shfl(at.page, tok) * a.page_bytes +
               (uint64_t)(uint32_t)((t0 + tok) & p.pmask) * a.row_bytes - (uint64_t)((tok & 15) * a.row_bytes);
      };
      const int r = lane / St::CH;
#pragma unroll 1
      for (int i = 0; i < 32 / St::RPL; i++) {
        const int kt = i * St::RPL + r, half = kt & 15, vt = (kt & 16) + 4 * (half & 3) + (half >> 2);
        load_lds16(klds + i * 1024, k + row(kt) + (KPH == 2 && (i & 1) ? koff[KPH - 1] : koff[0]));
        load_lds16(vlds + i * 1024, v + row(vt) + voff + (DP == 256 ? (i & 1) * 2 * a.row_bytes : 0));
      }
      const int st = DP == 256 ? lane >> 2 : (lane & 31) >> 1;
#pragma unroll 1
      for (int h = 0; h < 2; h++) {
        const uint64_t off = row(16 * h + st);
        load_lds4(slds + h * 2 * St::SCALES, sbase + off + soff);
        if constexpr (DP == 256) load_lds4(slds + h * 2 * St::SCALES + St::SCALES, v + off + soff);
      }
    }
  }
};

// Scores of a tile: S^T = K Q^T.
template <int DP, int RT>
__device__ __forceinline__ void scores(const Wave<DP, RT>& w, const Head<DP>& hd, const Nibbles& nb, const char* stage,
                                       f4 (&s)[RT][2]) {
  using St = Stage<DP>;
  constexpr int KS = DP / 32;
#pragma unroll
  for (int r = 0; r < RT; r++) s[r][0] = s[r][1] = f4{0, 0, 0, 0};
  uint32_t k[2][KS];
  uint16_t ks[2][DP == 256 ? 2 : 1];
#pragma unroll
  for (int sub = 0; sub < 2; sub++) {
    const char* at = stage + sub * 16 * St::ROW + hd.kread;
    if constexpr (DP == 64) {
      const uint2 x = *(const uint2*)at;
      k[sub][0] = x.x;
      k[sub][1] = x.y;
    } else {
#pragma unroll
      for (int j = 0; j < KS / 4; j++) {
        // chunk 2 g + 1 of 8 is at chunk 2 g's position ^ 1
        const u4 x = *(const u4*)(stage + sub * 16 * St::ROW + (hd.kread ^ (j * 16)));
#pragma unroll
        for (int e = 0; e < 4; e++) k[sub][4 * j + e] = x[e];
      }
    }
    const char* sc = stage + 2 * St::CODES + sub * 2 * St::SCALES + hd.kscale;
    ks[sub][0] = *(const uint16_t*)sc;
    if constexpr (DP == 256) ks[sub][1] = *(const uint16_t*)(sc + hd.kstep);
  }
  // a fence for the scheduler behind each step, which else makes all numbers first and runs out of registers
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < KS; i++) {
#pragma unroll
    for (int sub = 0; sub < 2; sub++) {
      const h8 x = nb.numbers(k[sub][i], both(ks[sub][DP == 256 ? i / 4 : 0]));
#pragma unroll
      for (int r = 0; r < RT; r++) s[r][sub] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, w.q[r][i], s[r][sub], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Before the values of a tile of which some token does not exist or some query does not see
// some token: a number there that is not finite must not meet the zero weight of such a
// query.  In the stage, scales of tokens that do not exist become 0, and so do those that are
// no finite number, and codes whose number is none; returns whether there was such a number:
// add_odd() gives it to the queries that see it.
template <int DP>
__device__ __forceinline__ bool clean_values(const QuantAttn& a, int head, char* stage, uint32_t alive) {
  using St = Stage<DP>;
  const int lane = rare_lane(), tok = lane & 31, r = tok & 15, odd = (head * a.groups) & 1;
  uint16_t* scale = (uint16_t*)(stage + 2 * St::CODES + ((tok >> 4) * 2 + 1) * St::SCALES + r * St::WIN) + odd;
  uint32_t* codes = (uint32_t*)(stage + St::CODES + ((tok >> 4) * 16 + 4 * (r & 3) + (r >> 2)) * St::ROW);
  const bool there = (alive >> tok) & 1;
  bool found = false;
#pragma unroll 1
  for (int j = lane >> 5; j < a.groups; j += 2) {
    const uint16_t bits = scale[j], size = bits & 0x7FFF;
    if (there && size <= 0x6FFE) continue;  // 8 s is finite
    if (!there || size >= 0x7C00) {
      scale[j] = 0;
      if (DP == 64) scale[j ^ 2] = 0;  // the window is one word twice
      found |= there;
      continue;
    }
    const float s = half_bits_to_float(bits);
#pragma unroll 1
    for (int i = 0; i < 32; i++) {
      const uint32_t w = codes[j * 4 + i / 8];
      const float x = (float)(_Float16)((float)((int)(w >> 4 * (i % 8) & 15) - 8) * s);
      if (x - x == 0.0f) continue;
      codes[j * 4 + i / 8] = (w & ~(15u << 4 * (i % 8))) | 8u << 4 * (i % 8);
      found = true;
    }
  }
  wait_lds();
  return __any(found);
}

// o += V^T P^T.  Row n of block b of V^T is channel b of the lane's, so that a lane's
// channels are neighbours in its word; its tokens come together two at a time.
template <int DP, int RT>
__device__ __forceinline__ void values(Wave<DP, RT>& w, const Head<DP>& hd, const Nibbles& nb, const char* stage,
                                       const h8 (&p)[RT]) {
  using St = Stage<DP>;
  constexpr int VW = DP == 256 ? 2 : 1, HALVES = DP == 64 ? 1 : 2;  // words of a lane, halves of a word
  uint32_t x[8][VW];
  union { s4 t[2]; h2 s[4]; } sc;  // scales of tokens 4 g .. + 3, 16 + 4 g .. + 3
#pragma unroll
  for (int sub = 0; sub < 2; sub++) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const char* at = stage + St::CODES + sub * 16 * St::ROW + i * 4 * St::ROW + hd.vread;
      if constexpr (VW == 2) {
        const uint2 y = *(const uint2*)at;
        x[4 * sub + i][0] = y.x;
        x[4 * sub + i][1] = y.y;
      } else {
        x[4 * sub + i][0] = *(const uint32_t*)at;
      }
    }
    sc.t[sub] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s4*)(stage + 2 * St::CODES + (2 * sub + 1) * St::SCALES + hd.vscale));
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int y = 0; y < VW * HALVES; y++) {  // 4 channels: bytes y % 2 and 2 + y % 2 of words y / 2
    union { uint32_t u[4]; h8 h; } v[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {  // tokens 4 g + 2 j, + 1 (j < 2), 16 + 4 g + 2 (j - 2), + 1
      const uint32_t w0 = x[2 * j][y / HALVES], w1 = x[2 * j + 1][y / HALVES];
      const uint32_t sel = DP == 64 ? hd.bytes : 0x0C040C00u + (y & 1) * 0x00010001u;
      const uint32_t even = __builtin_amdgcn_perm(w1, w0, sel), odd = __builtin_amdgcn_perm(w1, w0, sel + 0x00020002u);
      v[0].u[j] = __builtin_bit_cast(uint32_t, nb.get<false>(even) * sc.s[j]);
      v[1].u[j] = __builtin_bit_cast(uint32_t, nb.get<false>(odd) * sc.s[j]);
      v[2].u[j] = __builtin_bit_cast(uint32_t, nb.get<true>(even) * sc.s[j]);
      v[3].u[j] = __builtin_bit_cast(uint32_t, nb.get<true>(odd) * sc.s[j]);
    }
#pragma unroll
    for (int b = 0; b < 4; b++)
#pragma unroll
      for (int r = 0; r < RT; r++)
        w.o[r][y * 4 + b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[b].h, p[r], w.o[r][y * 4 + b], 0, 0, 0);
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
constexpr int kStages = 2;
template <int DP>
struct QuantShared {
  static constexpr int kWaves = kBlock / 64;
  __attribute__((aligned(1024))) char stage[kWaves][kStages][Stage<DP>::BYTES];  // then the sums of the waves
  int32_t list[kList];
  float m[kWaves][32], l[kWaves][32], scale[kWaves][32];
  uint32_t odd;  // values() found something
  uint32_t bad;  // a page met so far is outside the pool
};
static_assert(sizeof(QuantShared<128>) <= 160 * 1024 / 4, "four workgroups a compute unit");

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
  const int tid = rare_thread();
  row1 = min(row1, it.rows);
#pragma unroll 1
  for (int range = 0; range < ranges; range++) {
    const Item cur = range_of(it, ranges, range);
    const Split sp = split_of(a, cur);
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
__device__ __forceinline__ void run_few(const A& a, const Item& it, QuantShared<DP>& sh) {
  constexpr int kWaves = kBlock / 64;
  using W = Wave<DP, RT>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ranges = ranges_of(a, it);
  const int turn = kWaves / it.heads;  // waves of a head
  const int head = it.head + wave / turn;
  const float c = log2_scale(a);
  const int row_tiles = (it.rows + 16 * RT - 1) / (16 * RT);
  const int list_tiles = (int)((int64_t)(kList - 1) * a.P / kTile) - 1;
  {
    const Split sp = split_of(a, it);
    if (!a.direct && it.split >= sp.used) return;
  }
  const uint32_t lds = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char*)sh.stage[wave][0]);

  for (int rt = it.row_tile; rt < row_tiles; rt += it.row_tiles) {
    const Head<DP> hd(a, head);
    const Nibbles nb;
    W w;
    w.clear();
    w.template load_queries<true>(a, it, head, rt * 16 * RT);
    if (threadIdx.x == 0) sh.odd = sh.bad = 0;
#pragma unroll 1
    for (int range = 0; range < ranges; range++) {
      const Item cur = range_of(it, ranges, range);
      const Split sp = split_of(a, cur);
      if (cur.split >= sp.used) continue;
      const int first = sp.tile0 + cur.split * sp.per, last = min(first + sp.per, sp.tile0 + sp.tiles);
      const int min_lim = row_lim(a, cur, rt * 16 * RT);
      // tiles behind this one nobody of these rows sees
      const int end = min(last, (row_lim(a, cur, (rt + 1) * 16 * RT - 1) + kTile - 1) / kTile);
      for (int base = first; base < end; base += list_tiles) {
        const int stop = min(base + list_tiles, end);
        const int b0 = max(base * kTile, cur.lo) >> a.shift, b1 = (min(stop * kTile, cur.hi) - 1) >> a.shift;
        __syncthreads();  // the list is free
        for (int i = rare_thread(); i <= b1 - b0; i += kBlock) {
          const int page = a.tables[(int64_t)cur.trow * a.B + b0 + i];
          const bool ok = page >= 0 && page < a.N;
          sh.list[i] = ok ? page : -1;
          if (!ok) sh.bad = 1;
        }
        __syncthreads();
        // tokens that exist for this stretch lie in its blocks
        const Pages pages{sh.list, b0, max(base * kTile, cur.lo), min(stop * kTile, cur.hi), a.shift, a.P - 1};
        At at{0, 0}, next_at{0, 0};
        int tile = base + wave % turn, slot = 0;
        if (tile < stop) {
          at = find(pages, tile * kTile);
          hd.load(a, pages, at, tile * kTile, lds);
        }
        for (; tile < stop; tile += turn, slot ^= 1, at = next_at) {
          const int next = tile + turn;
          if (next < stop) {
            next_at = find(pages, next * kTile);
            wait_lds();  // the stage that is filled now has been read
            hd.load(a, pages, next_at, next * kTile, lds + (slot ^ 1) * Stage<DP>::BYTES);
            wait_loads<Stage<DP>::LOADS>();
          } else {
            wait_loads<0>();
          }
          char* stage = sh.stage[wave][slot];
          f4 s[RT][2];
          h8 p[RT];
          float mx[RT];
          scores(w, hd, nb, stage, s);
          const bool all = at.alive == 0xFFFFFFFFu && (tile + 1) * kTile <= min_lim;
          if (!all) mask_scores<DP, RT>(a, cur, rt * 16 * RT, s, tile * kTile, at.alive);
          const bool raise = w.peaks(s, c, mx);
          w.reference(raise, mx, c);
          w.weights(s, c, p);
          if (!all && clean_values<DP>(a, head, stage, at.alive)) sh.odd = 1;
          values(w, hd, nb, stage, p);
        }
        wait_lds();
      }
    }
    // the waves' sums together, against the largest reference exponent
    const int tid = rare_thread(), n = tid & 15, g = (tid & 63) >> 4;
#pragma unroll
    for (int r = 0; r < RT; r++) {
      const float l = w.sum(r);
      if (g == 0) {
        sh.m[wave][r * 16 + n] = w.m[r];
        sh.l[wave][r * 16 + n] = l;
      }
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
    // 4-channel quads of a row, rotated by row; the lane's channels are neighbours, of each row 4 g + i of
    // the products' results one, whose lane says which
    constexpr int kQuads = DP / 4;
    static_assert(sizeof(sh.stage) >= (size_t)kWaves * 16 * kQuads * 16, "room for the sums");
    f4* sums = (f4*)sh.stage;
#pragma unroll 1
    for (int r = 0; r < RT; r++) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int ch = __shfl(hd.channel, 4 * g + i);
#pragma unroll
        for (int b = 0; b < W::NB; b += 4) {
          f4 x = r == 0 ? f4{w.o[0][b][i], w.o[0][b + 1][i], w.o[0][b + 2][i], w.o[0][b + 3][i]}
                        : f4{w.o[RT - 1][b][i], w.o[RT - 1][b + 1][i], w.o[RT - 1][b + 2][i], w.o[RT - 1][b + 3][i]};
          if (ch < a.d) sums[(wave * 16 + n) * kQuads + (((ch + b) / 4 + n) & (kQuads - 1))] = x;
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int i = tid; i < it.heads * 16 * kQuads; i += kBlock) {
        const int quad = i % kQuads, x = i / kQuads % 16, hh = i / (16 * kQuads), w0 = hh * turn;
        const int ch = quad * 4, row = r * 16 + x, gr = rt * 16 * RT + row;
        if (gr >= it.rows || ch >= a.d) continue;
        f4 sum{0, 0, 0, 0};
#pragma unroll
        for (int y = 0; y < kWaves; y++) {
          const int of = (w0 + y) % kWaves;
          const float f = sh.scale[of][row];
          const f4 part = sums[(of * 16 + x) * kQuads + ((quad + x) & (kQuads - 1))];
          if (y < turn) sum += f * part;
        }
        if (a.direct) store_out(out_at(a, it, it.head + hh, gr) + ch, quotient_of(sum, sh.m[w0][row]));
        else *(f4*)(a.part + part_at(a, it, it.head + hh, gr) * a.d + ch) = sum;
      }
    }
    __syncthreads();
    if (sh.odd)
      add_odd(a, it, ranges, rt * 16 * RT, (rt + 1) * 16 * RT,
              [&](int h, int row) { return sh.m[(h - it.head) * turn][row - rt * 16 * RT] == 0.0f; });
    __syncthreads();  // m, l, scale and the sums are free
  }
}

// Workgroups on a compute unit, as LDS and registers allow.
__host__ __device__ constexpr int resident4(int dp, int rt) { return dp == 256 || (dp == 128 && rt == 2) ? 2 : rt == 2 ? 3 : 4; }

template <int DP, int RT, bool kDirect>
__global__ __launch_bounds__(kBlock, resident4(DP, RT)) void k_quant_attention(QuantCall<kDirect> a, int first, int end) {
  __shared__ QuantShared<DP> sh;
  // Neighbouring items, the kv heads of the same tokens, run on one of the 8 XCDs, to which
  // workgroups are dealt in turn: they share cache lines.
  const int b = blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
  for (int w = first + b; w < end; w += gridDim.x) {
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
  int dp, pre_splits, rest_splits, pre_least, rest_least, pre_tiles, rest_tiles, pre_mode, rest_mode, pre_groups,
      rest_heads;
  bool direct;
  size_t words;
};

template <int DP>
void launch(bool direct, int mode, const QuantAttn& a, int64_t first, int64_t end, hipStream_t st) {
  if (end <= first) return;
  const int grid = (int)std::min<int64_t>((end - first + 7) / 8 * 8, 1 << 22);  // a multiple of 8
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
  // Tiles of a split: so many that the launch, were all rows of the greatest length, is `slots`
  // workgroups, and at most kMostSplits splits, whose sums the join reads.
  constexpr int kMostSplits = 64, kRounds = 2;
  auto cut = [&](int64_t items, int64_t tokens, int64_t slots, int& splits, int& least) {
    const int64_t tiles = (tokens + kTile - 1) / kTile;
    int64_t per = (items * tiles + slots - 1) / slots;
    per = std::max<int64_t>({per, (tiles + kMostSplits - 1) / kMostSplits, kLeast});
    splits = (int)std::max<int64_t>(1, (tiles + per - 1) / per);
    least = (int)std::min<int64_t>(per, 1 << 26);
  };
  auto heads = [&]() {
    int n = 1;
    while (n < 4 && kv % (2 * n) == 0) n *= 2;
    return n;
  };
  p.rest_heads = heads();
  const int64_t slots = 256 * resident4(p.dp, p.rest_mode + 1);
  const int64_t own = std::max(0, x.max_len - (shared ? x.max_prefix : 0));
  cut((int64_t)std::max(1, x.n_seqs) * kv / p.rest_heads * p.rest_tiles, own, kRounds * slots, p.rest_splits, p.rest_least);
  p.pre_splits = 0;
  p.pre_least = kLeast;
  if (x.n_groups)
    cut((int64_t)x.n_groups * kv * p.pre_tiles, shared ? x.max_prefix : 0, slots, p.pre_splits, p.pre_least);
  // Sharing saves (sequences - 1) times the prefix and costs a second kernel and its
  // start, about 5 us: not for little.
  const int64_t saved = shared ? (int64_t)x.n_seqs * x.max_prefix * c.channels * 4 : 0;
  int all = 1, some = 1;
  cut((int64_t)std::max(1, x.n_seqs) * kv / p.rest_heads * p.rest_tiles, x.max_len, kRounds * slots, all, some);
  p.direct = saved <= (int64_t)16 << 20 && x.max_prefix <= 512 && all == 1;
  if (p.direct) {
    p.pre_groups = 0;
    p.pre_splits = 0;
    p.rest_splits = 1;
    p.rest_least = 1;
    p.words = 4;
    return p;
  }
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
              (uint32_t)r.row * (uint32_t)c->page_tokens, p.pre_least, p.rest_least};
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
