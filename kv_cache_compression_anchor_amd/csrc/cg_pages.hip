// Pages of a cache: copying, reserving and writing new tokens, forking, freeing,
// compacting (include/cachegen.h, "Paged caches").
//
// Two kinds of work.  Bookkeeping (who gets which page) is a handful of prefix
// sums over the requests and over refs; each call does it in one workgroup of
// 1,024 threads, so that one launch suffices and page numbers do not depend on
// scheduling.  Its time is its chain of dependent loads and barriers: 5 to 11 us
// for up to 1,024 requests, 6,000 tokens and 16,384 pages; 88 us where the slots of
// 100,000 tokens are asked for and 1.9 ms for 2^21, which one workgroup finds one by
// one; 45 us for a compaction over 131,072 pages.  Moving K and V is a plain copy bound
// by HBM; it is cut into pieces spread over the chip.  Measured, counting bytes
// read and written: 96 pages of 32 layers x 16 tokens x 4,096 channels (1.6 GB)
// copied in 318 us, 5.1 TB/s; 5,850 tokens of 32 layers x 1,024 channels (1.5 GB)
// written in 297 us, 5.2 TB/s; 48 of 96 rows freed and 271 pages of the rest
// moved (1.1 GB) in 233 us, 4.9 TB/s; 64 forks of one row (a copy of 11 tokens
// each, 185 MB) in 25 us, 7.4 TB/s as their sources are read from the caches.  A
// large device-to-device copy reaches 4.7 TB/s here.
#include <algorithm>

#include "cg_hostapi.h"
#include "cg_internal.h"
#include "cg_paged.h"

namespace cg {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 1024;            // of a bookkeeping workgroup
constexpr int kWaves = kThreads / 64;
constexpr int kScanPages = 16 * kThreads; // pages of refs looked at per scan step
constexpr int kCopyThreads = 256;
// Units a copying workgroup moves per piece: four loads in flight a thread where there
// is enough to do, one where workgroups are scarce.
constexpr int kPieceMost = 4 * kCopyThreads, kPieceLeast = kCopyThreads;
constexpr uint32_t kBadPage = 2u, kRefused = 4u, kNoPages = 8u;  // status bits

struct Cache {  // the device side's view of cg_paged_cache
  int L, C, P, shift, N, R, B;
  char *k, *v;
  int32_t *tables, *lens, *refs;
  uint32_t* status;
};

// ---------------------------------------------------------------------------
// Prefix sums of a bookkeeping workgroup
// ---------------------------------------------------------------------------
__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }
__device__ __forceinline__ int below(uint64_t mask) {  // set bits below this lane
  return __popcll(mask & ((1ull << lane_id()) - 1));
}

struct ScanLds {
  uint32_t wave[kWaves];
};

// Sums stay at 2^32 - 1 once they are there: no pool has so many pages.
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// exclusive sum of one value per wave
__device__ __forceinline__ uint32_t wave_sums(uint32_t of_wave, ScanLds& s, uint32_t* total) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  __syncthreads();  // s is free again
  if (lane_id() == 0) s.wave[wave] = of_wave;
  __syncthreads();
  uint32_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; w++) {
    const uint32_t x = s.wave[w];
    if (w < wave) base = add(base, x);
    all = add(all, x);
  }
  *total = all;
  return base;
}

// Exclusive sum of one value per thread; *total receives the sum.  Within a wave by
// moves between lanes of the vector unit, a tenth of the latency of moves through LDS.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, ScanLds& s, uint32_t* total) {
  uint32_t inc = x;
#define FROM(ctrl, rows) add(inc, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)inc, ctrl, rows, 0xF, false))
  inc = FROM(0x111, 0xF);  // from 1, 2, 4 and 8 lanes below in a row of 16
  inc = FROM(0x112, 0xF);
  inc = FROM(0x114, 0xF);
  inc = FROM(0x118, 0xF);
  inc = FROM(0x142, 0xA);  // from the last lane of the row below to rows 1 and 3
  inc = FROM(0x143, 0xC);  // from lane 31 to rows 2 and 3
#undef FROM
  uint32_t before = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)inc, 0x138, 0xF, 0xF, false);  // of the lane below
  return add(wave_sums((uint32_t)__builtin_amdgcn_readlane((int)inc, 63), s, total), before);
}

// A wave's share of a scan step: 1,024 consecutive pages, 16 coalesced loads in flight
// (loads that are each under a condition wait for one another, 5 us in all: those past
// the end read the last count, which nobody looks at).
struct Counts {
  int32_t r[16];
  __device__ __forceinline__ static int page(int base, int i) {
    return base + (threadIdx.x >> 6) * 1024 + lane_id() + 64 * i;
  }
  __device__ __forceinline__ void load(const int32_t* refs, int base, int to) {
#pragma unroll
    for (int i = 0; i < 16; i++) r[i] = refs[min(page(base, i), to - 1)];
  }
};

// Calls f(page, rank) for those of a step's pages in [from, to) that are free (kFree) or
// in use (!kFree), rank in ascending order from `found` on; returns how many.
template <bool kFree, class F>
__device__ __forceinline__ int scan_step(const Counts& c, int base, int from, int to, int found, ScanLds& s, F f) {
  uint64_t hit[16];
  int n = 0;
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const int p = Counts::page(base, i);
    hit[i] = __ballot(p >= from && p < to && (kFree ? c.r[i] == 0 : c.r[i] > 0));
    n += __popcll(hit[i]);
  }
  uint32_t all;
  int rank = found + (int)wave_sums(n, s, &all);
#pragma unroll
  for (int i = 0; i < 16; i++) {
    if ((hit[i] >> lane_id()) & 1) f(Counts::page(base, i), rank + below(hit[i]));
    rank += __popcll(hit[i]);
  }
  return (int)all;
}

// The same for all steps of [from, to), until `limit` were found; returns how many
// there are up to where it stopped.  first: the first step's counts, loaded before.
template <bool kFree, class F>
__device__ int scan_pages(const int32_t* refs, const Counts& first, int from, int to, int limit, ScanLds& s, F f) {
  int found = 0;
  Counts c = first;
  for (int base = from; base < to && found < limit; base += kScanPages) {
    if (base != from) c.load(refs, base, to);
    found += scan_step<kFree>(c, base, from, to, found, s, f);
  }
  return found;
}
template <bool kFree, class F>
__device__ int scan_pages(const int32_t* refs, int from, int to, int limit, ScanLds& s, F f) {
  Counts c;
  if (from < to) c.load(refs, from, to);
  return scan_pages<kFree>(refs, c, from, to, limit, s, f);
}

// One bit per row of the cache (n_rows <= 65536).
constexpr int kRowWords = 65536 / 32;
__device__ __forceinline__ void clear_bits(uint32_t* b, int rows) {
  for (int i = threadIdx.x; i < (rows + 31) / 32; i += kThreads) b[i] = 0;
}
__device__ __forceinline__ bool test_bit(const uint32_t* b, int i) { return (b[i >> 5] >> (i & 31)) & 1; }
__device__ __forceinline__ bool set_bit(uint32_t* b, int i) {  // whether it was set before
  return (atomicOr(&b[i >> 5], 1u << (i & 31)) >> (i & 31)) & 1;
}

__device__ __forceinline__ bool row_ok(const Cache& c, int r) { return r >= 0 && r < c.R; }
__device__ __forceinline__ bool page_ok(const Cache& c, int p) { return p >= 0 && p < c.N; }
__device__ __forceinline__ bool len_ok(const Cache& c, int64_t n) {
  return n >= 0 && n <= (int64_t)c.B << c.shift;
}
__device__ __forceinline__ int blocks_of(const Cache& c, int64_t n) {
  return (int)((n + c.P - 1) >> c.shift);
}
__device__ __forceinline__ int32_t& entry(const Cache& c, int row, int b) {
  return c.tables[(int64_t)row * c.B + b];
}

// largest i in [0, n) with a[i] <= x, or -1
__device__ __forceinline__ int last_at_most(const int32_t* a, int n, int x) {
  int lo = -1, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a[m] <= x) lo = m; else hi = m;
  }
  return lo;
}

// a / b of numbers that mostly fit 32 bits
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// ---------------------------------------------------------------------------
// Moving rows of pages
// ---------------------------------------------------------------------------
// Piece `piece` of the copy of the first `units` units (of sizeof(U) bytes) of
// page src to page dst in all layers of both pools, by kCopyThreads threads; the units
// of the (kv, layer)s are numbered through.  Four loads are in flight per thread.
template <class U>
__device__ __forceinline__ void copy_piece(const Cache& c, int src, int dst, uint32_t units,
                                           int64_t piece, int piece_units) {
  const int64_t all = (int64_t)2 * c.L * units;
  const int64_t first = piece * piece_units;
  const int64_t page_bytes = (int64_t)c.P * c.C * 2;
  const uint32_t n = (uint32_t)(all - first < piece_units ? all - first : piece_units);
  // a 64-bit division is a microsecond of latency
  const uint32_t sl0 = all >> 32 ? (uint32_t)(first / units) : (uint32_t)first / units;
  const uint32_t u0 = (uint32_t)(first - (int64_t)sl0 * units);
  const int64_t from = src * page_bytes, to = dst * page_bytes;
  auto place = [&](uint32_t e) {  // of unit u0 + e in page 0
    const uint32_t more = e / units, u = e - more * units, sl = sl0 + more;
    const bool v = sl >= (uint32_t)c.L;
    return (v ? c.v : c.k) + (int64_t)(v ? sl - c.L : sl) * c.N * page_bytes + (int64_t)u * sizeof(U);
  };
  uint32_t i = threadIdx.x % kCopyThreads;
  for (; i + 3 * kCopyThreads < n; i += 4 * kCopyThreads) {
    char *a0 = place(u0 + i), *a1 = place(u0 + i + kCopyThreads), *a2 = place(u0 + i + 2 * kCopyThreads),
         *a3 = place(u0 + i + 3 * kCopyThreads);
    const U x0 = *(const U*)(a0 + from), x1 = *(const U*)(a1 + from), x2 = *(const U*)(a2 + from),
            x3 = *(const U*)(a3 + from);
    *(U*)(a0 + to) = x0;
    *(U*)(a1 + to) = x1;
    *(U*)(a2 + to) = x2;
    *(U*)(a3 + to) = x3;
  }
  for (; i < n; i += kCopyThreads) {
    char* a0 = place(u0 + i);
    *(U*)(a0 + to) = *(const U*)(a0 + from);
  }
}

__host__ __device__ __forceinline__ int64_t pieces_of(int L, int64_t units, int piece) {
  return (2 * (int64_t)L * units + piece - 1) / piece;
}

// Pair i is copied unless its dst is named twice or its src is a dst: every
// workgroup looks through the lists for its own pair, n / 256 pairs a thread,
// which needs no workspace and no second launch.  Up to kFewPairs pairs, where the
// list is no longer than a piece: 4,000 pages of 16 x 32 KB take 834 us so and 863 by
// runs of pairs (below), 8,000 take 1,761 and 1,708, 8,000 pages of 4 x 4 KB 57 and
// 41, a million of 4 x 256 B 327 ms and 1.9.
constexpr int kFewPairs = 4096;
template <class U>
__global__ __launch_bounds__(kCopyThreads) void k_pages_copy(Cache c, int n, const int32_t* src,
                                                             const int32_t* dst, int64_t pieces,
                                                             int piece_units) {
  for (int64_t w = blockIdx.x; w < n * pieces; w += gridDim.x) {
    const int i = (int)quotient(w, pieces);
    const int s = src[i], d = dst[i];
    bool clash = false;
    for (int j = threadIdx.x; j < n; j += kCopyThreads) {
      const int o = dst[j];
      clash |= o == s || (o == d && j != i);
    }
    clash = __syncthreads_or(clash);
    if (!page_ok(c, s) || !page_ok(c, d)) {
      if (threadIdx.x == 0) atomicOr(c.status, kBadPage);
    } else if (clash) {
      if (threadIdx.x == 0) atomicOr(c.status, kRefused);
    } else {
      copy_piece<U>(c, s, d, (uint32_t)((int64_t)c.P * c.C * 2 / sizeof(U)), w - i * pieces, piece_units);
    }
  }
}

// More pairs: a workgroup takes a run of them and looks through dst once for all of
// them, up to kRunPairs at a time, counting how often each of their pages is named
// there: so the lists are read n / kRunPairs times in all, or as often as there are
// workgroups, and not once for every piece.
constexpr int kRunThreads = 1024, kRuns = 512;  // two workgroups a compute unit, 68 KB of LDS each
constexpr int kRunPairs = 4096, kPageSlots = 4 * kRunPairs;

// Pages by open addressing; at most half of the slots are taken, so a search ends.
struct PageTable {
  // 0: free; page + 1, whether dst names it, whether it does so again
  static constexpr uint32_t kPage = (1u << 25) - 1, kOnce = 1u << 30, kTwice = 1u << 31;
  uint32_t slot[kPageSlots];

  __device__ __forceinline__ static uint32_t place(int page) { return (uint32_t)page * 2654435761u >> 18; }
  static_assert(kPageSlots == 1 << (32 - 18), "place() gives a slot");
  __device__ __forceinline__ void insert(int page) {
    for (uint32_t i = place(page);; i = (i + 1) % kPageSlots) {
      const uint32_t x = atomicCAS(&slot[i], 0u, (uint32_t)page + 1);
      if (x == 0 || x == (uint32_t)page + 1) return;
    }
  }
  // the slot of a page, -1 if it has none
  __device__ __forceinline__ int find(int page, uint32_t* x) const {
    for (uint32_t i = place(page);; i = (i + 1) % kPageSlots) {
      *x = slot[i];
      if (*x == 0) return -1;
      if ((*x & kPage) == (uint32_t)page + 1) return (int)i;
    }
  }
  __device__ __forceinline__ void count(int page) {
    uint32_t x;
    const int i = find(page, &x);
    if (i >= 0 && !(x & kTwice) && (atomicOr(&slot[i], kOnce) & kOnce)) atomicOr(&slot[i], kTwice);
  }
};

template <class U>
__global__ __launch_bounds__(kRunThreads, 8) void k_pages_copy_many(Cache c, int n, const int32_t* src,
                                                                    const int32_t* dst, int run,
                                                                    int64_t pieces, int piece_units) {
  __shared__ PageTable table;
  __shared__ uint8_t copied[kRunPairs];  // whether the pair is
  const int64_t begin = (int64_t)blockIdx.x * run;
  const int end = (int)(begin + run < n ? begin + run : n);
  for (int i0 = (int)(begin < n ? begin : n); i0 < end; i0 += kRunPairs) {
    const int pairs = min(kRunPairs, end - i0);
    __syncthreads();  // the tables are free
    for (int i = threadIdx.x; i < kPageSlots; i += kRunThreads) table.slot[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += kRunThreads) {
      const int s = src[i0 + i], d = dst[i0 + i];
      const bool ok = page_ok(c, s) && page_ok(c, d);
      copied[i] = ok;
      if (ok) {
        table.insert(s);
        table.insert(d);
      } else {
        atomicOr(c.status, kBadPage);
      }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += 4 * kRunThreads) {
      int page[4];  // loads in flight together
#pragma unroll
      for (int k = 0; k < 4; k++) page[k] = dst[min(j + k * kRunThreads, n - 1)];
#pragma unroll
      for (int k = 0; k < 4; k++)
        if (j + k * kRunThreads < n && page_ok(c, page[k])) table.count(page[k]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += kRunThreads) {
      if (!copied[i]) continue;
      uint32_t s, d;
      table.find(src[i0 + i], &s);
      table.find(dst[i0 + i], &d);
      if ((s & PageTable::kOnce) || (d & PageTable::kTwice)) {
        copied[i] = 0;
        atomicOr(c.status, kRefused);
      }
    }
    __syncthreads();
    const uint32_t units = (uint32_t)((int64_t)c.P * c.C * 2 / sizeof(U));
    for (int64_t w = threadIdx.x / kCopyThreads; w < pairs * pieces; w += kRunThreads / kCopyThreads) {
      const int i = (int)quotient(w, pieces);
      if (copied[i]) copy_piece<U>(c, src[i0 + i], dst[i0 + i], units, w - i * pieces, piece_units);
    }
  }
}

// Up to kFew requests, one a thread, and their dealt pages are kept in registers and
// LDS: a bookkeeping kernel's time is its chain of dependent global loads, and searches
// and lists in global memory made most of it.
constexpr int kFew = kThreads, kFewPages = 4096;

// ---------------------------------------------------------------------------
// Reserve
// ---------------------------------------------------------------------------
// Slots of tokens [t0, t1): the request by binary search in starts, the page
// from the row's table.  Runs behind the tables' and lens' update.
__device__ void fill_slots(const Cache& c, int n, const int32_t* rows, const int32_t* starts,
                           const int32_t* ok, int64_t* slots, int t0, int t1, int step) {
  for (int t = t0; t < t1; t += step) {
    int64_t slot = -1;
    const int i = last_at_most(starts, n, t);
    if (i >= 0 && t < starts[i + 1] && ok[i]) {
      const int row = rows[i];
      const int64_t pos = (int64_t)c.lens[row] - (starts[i + 1] - t);
      const int page = entry(c, row, (int)(pos >> c.shift));
      if (page_ok(c, page))
        slot = ((int64_t)page << c.shift) + (pos & (c.P - 1));
      else
        atomicOr(c.status, kBadPage);
    }
    slots[t] = slot;
  }
}

__global__ __launch_bounds__(kThreads) void k_reserve(Cache c, int n, const int32_t* rows,
                                                      const int32_t* starts, int n_tokens,
                                                      int64_t* slots, int32_t* cum, int32_t* ok,
                                                      int32_t* list) {
  __shared__ ScanLds s;
  __shared__ uint32_t seen[kRowWords], twice[kRowWords];
  clear_bits(seen, c.R);
  clear_bits(twice, c.R);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (row_ok(c, rows[i]) && set_bit(seen, rows[i])) set_bit(twice, rows[i]);
  __syncthreads();
  // what each request needs, and where its pages start in the dealt list
  constexpr int64_t kMany = 1 << 30;  // sums are cut there: no pool has so many pages
  int64_t sum = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + threadIdx.x;
    int need = 0, good = 0;
    if (i < n) {
      const int row = rows[i], a = starts[i], b = starts[i + 1];
      if (row_ok(c, row) && !test_bit(twice, row) && a >= 0 && a <= b && b <= n_tokens) {
        const int64_t len = c.lens[row];
        if (len_ok(c, len) && len_ok(c, len + (b - a))) {
          good = 1;
          need = blocks_of(c, len + (b - a)) - blocks_of(c, len);
        }
      }
      if (!good) atomicOr(c.status, kRefused);
    }
    uint32_t all;
    const int64_t at = sum + block_scan(need, s, &all);
    if (i < n) {
      cum[i] = (int)(at < kMany ? at : kMany);
      ok[i] = good;
    }
    sum += all;
  }
  const int total = (int)(sum < kMany ? sum : kMany);
  if (threadIdx.x == 0) cum[n] = total;
  __syncthreads();
  const int found = total ? scan_pages<true>(c.refs, 0, c.N, total, s,
                                             [&](int page, int rank) {
                                               if (rank < total) list[rank] = page;
                                             })
                          : 0;
  const int have = min(found, total);
  __syncthreads();
  for (int r = threadIdx.x; r < have; r += kThreads) {
    const int i = last_at_most(cum, n, r);  // the last of equal ones: the request that needs pages
    if (cum[i + 1] <= have) {
      const int row = rows[i];
      entry(c, row, blocks_of(c, c.lens[row]) + (r - cum[i])) = list[r];
      c.refs[list[r]] = 1;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    if (!ok[i]) continue;
    if (cum[i + 1] > cum[i] && cum[i + 1] > have) {
      ok[i] = 0;
      atomicOr(c.status, kNoPages);
    } else {
      c.lens[rows[i]] += starts[i + 1] - starts[i];
    }
  }
  if (!slots) return;
  __syncthreads();
  fill_slots(c, n, rows, starts, ok, slots, threadIdx.x, n_tokens, kThreads);
}

__global__ __launch_bounds__(kThreads) void k_reserve_few(Cache c, int n, const int32_t* rows,
                                                          const int32_t* starts, int n_tokens,
                                                          int64_t* slots, int32_t* list) {
  __shared__ ScanLds s;
  __shared__ uint32_t seen[kRowWords], twice[kRowWords];
  __shared__ int32_t cum[kFew + 1], start[kFew + 1], old_len[kFew], old_page[kFew], of_row[kFew], dealt[kFewPages];
  const int i = threadIdx.x;
  // all loads are made without conditions, which would have them wait for one another
  const int ic = min(i, n - 1), some_row = rows[ic], a = starts[ic], b = starts[ic + 1];
  Counts counts;
  counts.load(c.refs, 0, c.N);
  clear_bits(seen, c.R);
  clear_bits(twice, c.R);
  const int row = i < n ? some_row : -1;
  const bool known = row_ok(c, row);
  const int some_len = c.lens[known ? row : 0], len = known ? some_len : -1;
  __syncthreads();
  if (known && set_bit(seen, row)) set_bit(twice, row);
  const bool fits = known && a >= 0 && a <= b && b <= n_tokens && len_ok(c, len) &&
                    len_ok(c, (int64_t)len + (b - a));
  const int last = entry(c, fits ? row : 0, fits && len ? blocks_of(c, len) - 1 : 0);
  __syncthreads();
  const bool good = fits && !test_bit(twice, row);
  if (i < n && !good) atomicOr(c.status, kRefused);
  const int need = good ? blocks_of(c, (int64_t)len + (b - a)) - blocks_of(c, len) : 0;
  constexpr uint32_t kMany = 1 << 30;  // sums are cut there: no pool has so many pages
  uint32_t sum;
  const uint32_t at = block_scan(need, s, &sum);
  const int total = (int)(sum < kMany ? sum : kMany);
  if (i < n) {
    cum[i] = (int)(at < kMany ? at : kMany);
    start[i] = a;
    of_row[i] = row;
    old_page[i] = last;
    if (i == n - 1) {
      cum[n] = total;
      start[n] = b;
    }
  }
  int32_t* pages = total <= kFewPages ? dealt : list;
  const int found = total ? scan_pages<true>(c.refs, counts, 0, c.N, total, s,
                                             [&](int page, int rank) {
                                               if (rank < total) pages[rank] = page;
                                             })
                          : 0;
  const int have = min(found, total);
  if (i < n) {
    const bool granted = good && (need == 0 || (int64_t)at + need <= have);
    old_len[i] = granted ? len : -1;
    if (granted) c.lens[row] = len + (b - a);
    else if (good) atomicOr(c.status, kNoPages);
  }
  __syncthreads();
  for (int r = i; r < have; r += kThreads) {
    const int j = last_at_most(cum, n, r);  // the last of equal ones: the request that needs pages
    if (old_len[j] < 0) continue;
    const int page = pages[r];
    entry(c, of_row[j], blocks_of(c, old_len[j]) + (r - cum[j])) = page;
    c.refs[page] = 1;
  }
  for (int t = i; slots && t < n_tokens; t += kThreads) {
    int64_t slot = -1;
    const int j = last_at_most(start, n, t);
    if (j >= 0 && t < start[j + 1] && old_len[j] >= 0) {
      const int64_t pos = (int64_t)old_len[j] + (t - start[j]);
      const int blk = (int)(pos >> c.shift), old = blocks_of(c, old_len[j]);
      const int page = blk < old ? old_page[j] : pages[cum[j] + blk - old];
      if (page_ok(c, page))
        slot = ((int64_t)page << c.shift) + (pos & (c.P - 1));
      else
        atomicOr(c.status, kBadPage);
    }
    slots[t] = slot;
  }
}

// ---------------------------------------------------------------------------
// Write
// ---------------------------------------------------------------------------
// A workgroup writes `tile` tokens of one (kv, layer): a token's row is `units`
// units, contiguous on both sides.
template <class U>
__global__ __launch_bounds__(kCopyThreads) void k_write(Cache c, int layer0, int n_layers,
                                                        int n_tokens, const int64_t* slots,
                                                        const char* k_new, const char* v_new,
                                                        int64_t token_bytes, int64_t layer_bytes,
                                                        uint32_t units, int tile) {
  const int sl = blockIdx.y, l = sl < n_layers ? sl : sl - n_layers;
  const char* from = (sl < n_layers ? k_new : v_new) + l * layer_bytes;
  const int64_t row_bytes = (int64_t)c.C * 2;
  char* to = (sl < n_layers ? c.k : c.v) + (int64_t)(layer0 + l) * c.N * c.P * row_bytes;
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  const uint32_t nt = (uint32_t)(n_tokens - t0 < tile ? n_tokens - t0 : tile);
  const int64_t cap = (int64_t)c.N << c.shift;
  for (uint32_t e = threadIdx.x; e < nt * units; e += kCopyThreads) {
    const uint32_t t = e / units, u = e % units;
    const int64_t slot = slots[t0 + t];
    if (slot >= 0 && slot < cap)
      *(U*)(to + slot * row_bytes + (int64_t)u * sizeof(U)) =
          *(const U*)(from + (t0 + t) * token_bytes + (int64_t)u * sizeof(U));
    else if (slot != -1 && u == 0)
      atomicOr(c.status, kBadPage);
  }
}

// ---------------------------------------------------------------------------
// Fork
// ---------------------------------------------------------------------------
// aux[3 i ..]: the parent's partly filled page, the child's page, rows in use
__global__ __launch_bounds__(kThreads) void k_fork_plan(Cache c, int n, const int32_t* parents,
                                                        const int32_t* children, int32_t* ok,
                                                        int32_t* cum, int32_t* aux,
                                                        int32_t* list) {
  __shared__ ScanLds s;
  __shared__ uint32_t kids[kRowWords], twice[kRowWords], olds[kRowWords];
  clear_bits(kids, c.R);
  clear_bits(twice, c.R);
  clear_bits(olds, c.R);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    if (row_ok(c, children[i]) && set_bit(kids, children[i])) set_bit(twice, children[i]);
    if (row_ok(c, parents[i])) set_bit(olds, parents[i]);
  }
  __syncthreads();
  int total = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + threadIdx.x;
    int need = 0, good = 0;
    if (i < n) {
      const int par = parents[i], kid = children[i];
      int part = 0, last = -1;
      if (row_ok(c, par) && row_ok(c, kid) && !test_bit(twice, kid) && !test_bit(olds, kid) &&
          c.lens[kid] == 0 && len_ok(c, c.lens[par])) {
        const int len = c.lens[par];
        good = 1;
        part = len & (c.P - 1);
        if (part) {
          last = entry(c, par, blocks_of(c, len) - 1);
          need = 1;
          if (!page_ok(c, last)) {
            good = need = 0;
            atomicOr(c.status, kBadPage);
          }
        }
      } else {
        atomicOr(c.status, kRefused);
      }
      aux[3 * i] = last;
      aux[3 * i + 2] = part;
    }
    uint32_t all;
    const int64_t at = block_scan(need, s, &all);
    if (i < n) {
      cum[i] = total + (int)at;
      ok[i] = good | need << 1;
    }
    total += (int)all;
  }
  const int found = total ? scan_pages<true>(c.refs, 0, c.N, total, s,
                                             [&](int page, int rank) {
                                               if (rank < total) list[rank] = page;
                                             })
                          : 0;
  const int have = min(found, total);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    if (!(ok[i] & 1)) continue;
    if ((ok[i] & 2) && cum[i] >= have) {
      ok[i] = 0;
      atomicOr(c.status, kNoPages);
      continue;
    }
    if (ok[i] & 2) {
      aux[3 * i + 1] = list[cum[i]];
      c.refs[list[cum[i]]] = 1;
    }
    c.lens[children[i]] = c.lens[parents[i]];
  }
}

__global__ __launch_bounds__(kThreads) void k_fork_plan_few(Cache c, int n, const int32_t* parents,
                                                            const int32_t* children, int32_t* ok,
                                                            int32_t* aux) {
  __shared__ ScanLds s;
  __shared__ uint32_t kids[kRowWords], twice[kRowWords], olds[kRowWords];
  __shared__ int32_t dealt[kFew];
  const int i = threadIdx.x;
  const int ic = min(i, n - 1), some_par = parents[ic], some_kid = children[ic];
  Counts counts;
  counts.load(c.refs, 0, c.N);
  clear_bits(kids, c.R);
  clear_bits(twice, c.R);
  clear_bits(olds, c.R);
  const int par = i < n ? some_par : -1, kid = i < n ? some_kid : -1;
  const bool known = row_ok(c, par) && row_ok(c, kid);
  const int some_len = c.lens[known ? par : 0], kid_len = c.lens[known ? kid : 0], len = known ? some_len : -1;
  __syncthreads();
  if (row_ok(c, kid) && set_bit(kids, kid)) set_bit(twice, kid);
  if (row_ok(c, par)) set_bit(olds, par);
  const bool fits = known && kid_len == 0 && len_ok(c, len);
  const int part = fits ? len & (c.P - 1) : 0;
  const int last = entry(c, part ? par : 0, part ? blocks_of(c, len) - 1 : 0);
  __syncthreads();
  bool good = fits && !test_bit(twice, kid) && !test_bit(olds, kid);
  if (i < n && !good) atomicOr(c.status, kRefused);
  if (good && part && !page_ok(c, last)) {
    good = false;
    atomicOr(c.status, kBadPage);
  }
  const int need = good && part;
  uint32_t total;
  const int at = (int)block_scan(need, s, &total);
  const int found = total ? scan_pages<true>(c.refs, counts, 0, c.N, (int)total, s,
                                             [&](int page, int rank) {
                                               if (rank < (int)total) dealt[rank] = page;
                                             })
                          : 0;
  __syncthreads();
  if (i >= n) return;
  if (need && at >= found) {
    good = false;
    atomicOr(c.status, kNoPages);
  }
  ok[i] = good;
  if (!good) return;
  aux[3 * i] = last;
  aux[3 * i + 1] = need ? dealt[at] : -1;
  aux[3 * i + 2] = part;
  if (need) c.refs[dealt[at]] = 1;
  c.lens[kid] = len;
}

// blockIdx.y 0: the child's table row and the counts; others: pieces of the copy
template <class U>
__global__ __launch_bounds__(kCopyThreads) void k_fork_copy(Cache c, const int32_t* parents,
                                                            const int32_t* children,
                                                            const int32_t* ok, const int32_t* aux,
                                                            int piece_units) {
  const int i = blockIdx.x;
  if (!(ok[i] & 1)) return;
  const int part = aux[3 * i + 2], to = aux[3 * i + 1];
  if (blockIdx.y == 0) {
    const int par = parents[i], kid = children[i];
    const int nblk = blocks_of(c, c.lens[par]);
    for (int b = threadIdx.x; b < nblk; b += kCopyThreads) {
      const bool own = part && b == nblk - 1;
      const int p = entry(c, par, b);
      entry(c, kid, b) = own ? to : p;
      if (own) continue;
      if (page_ok(c, p))
        atomicAdd(&c.refs[p], 1);
      else
        atomicOr(c.status, kBadPage);
    }
    return;
  }
  if (!part) return;
  const uint32_t units = (uint32_t)((int64_t)part * c.C * 2 / sizeof(U));
  const int64_t pieces = pieces_of(c.L, units, piece_units);
  for (int64_t w = blockIdx.y - 1; w < pieces; w += gridDim.y - 1)
    copy_piece<U>(c, aux[3 * i], to, units, w, piece_units);
}

// ---------------------------------------------------------------------------
// Free
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kCopyThreads) void k_free(Cache c, int n, const int32_t* rows) {
  const int i = blockIdx.x, row = rows[i];
  bool again = false;
  for (int j = threadIdx.x; j < i; j += kCopyThreads) again |= rows[j] == row;
  again = __syncthreads_or(again);
  if (again || !row_ok(c, row) || !len_ok(c, c.lens[row])) {
    if (threadIdx.x == 0) atomicOr(c.status, kRefused);
    return;
  }
  const int nblk = blocks_of(c, c.lens[row]);
  for (int b = threadIdx.x; b < nblk; b += kCopyThreads) {
    const int p = entry(c, row, b);
    entry(c, row, b) = -1;
    if (!page_ok(c, p)) {
      atomicOr(c.status, kBadPage);
    } else if (atomicSub(&c.refs[p], 1) <= 0) {  // counts that were wrong before stay at 0
      atomicAdd(&c.refs[p], 1);
      atomicOr(c.status, kRefused);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) c.lens[row] = 0;
}

// ---------------------------------------------------------------------------
// Compact
// ---------------------------------------------------------------------------
// ws[0] moves; from[j], to[j]: the j-th move; where[p - M]: move of page p
__global__ __launch_bounds__(kThreads) void k_compact_plan(Cache c, int32_t* live_out, int32_t* ws,
                                                           int32_t* to, int32_t* from) {
  __shared__ ScanLds s;
  const int live = scan_pages<false>(c.refs, 0, c.N, c.N, s, [](int, int) {});
  const int frees =
      scan_pages<true>(c.refs, 0, live, c.N, s, [&](int page, int rank) { to[rank] = page; });
  const int above = scan_pages<false>(c.refs, live, c.N, c.N, s,
                                      [&](int page, int rank) { from[rank] = page; });
  // as many as each other unless some count is negative
  const int moves = min(frees, above);
  if (frees != above && threadIdx.x == 0) atomicOr(c.status, kRefused);
  __syncthreads();
  for (int j = threadIdx.x; j < moves; j += kThreads) {
    c.refs[to[j]] = c.refs[from[j]];
    c.refs[from[j]] = 0;
  }
  if (threadIdx.x == 0) {
    ws[0] = moves;
    if (live_out) *live_out = live;
  }
}

// Up to one scan step of pages: refs are read once and the lists pass through LDS.
__global__ __launch_bounds__(kThreads) void k_compact_plan_few(Cache c, int32_t* live_out, int32_t* ws,
                                                               int32_t* to, int32_t* from) {
  __shared__ ScanLds s;
  __shared__ uint16_t below_live[kScanPages / 2], above_live[kScanPages / 2];
  static_assert(kScanPages <= 65536, "page numbers in 16 bits");
  Counts counts;
  counts.load(c.refs, 0, c.N);
  const int live = scan_step<false>(counts, 0, 0, c.N, 0, s, [](int, int) {});
  // no more than half of the pages can be free below the live count, or in use above it,
  // unless counts are negative: those further on are left where they are
  const int frees = scan_step<true>(counts, 0, 0, live, 0, s, [&](int page, int rank) {
    if (rank < kScanPages / 2) below_live[rank] = (uint16_t)page;
  });
  const int above = scan_step<false>(counts, 0, live, c.N, 0, s, [&](int page, int rank) {
    if (rank < kScanPages / 2) above_live[rank] = (uint16_t)page;
  });
  const int moves = min(min(frees, above), kScanPages / 2);
  if (frees != above && threadIdx.x == 0) atomicOr(c.status, kRefused);
  __syncthreads();
  for (int j = threadIdx.x; j < moves; j += kThreads) {
    const int a = above_live[j], b = below_live[j];
    to[j] = b;
    from[j] = a;
    c.refs[b] = c.refs[a];
    c.refs[a] = 0;
  }
  if (threadIdx.x == 0) {
    ws[0] = moves;
    if (live_out) *live_out = live;
  }
}

// Tables follow (an entry's move by binary search in the ascending `from`), then
// the pages are copied; both spread over a fixed grid, as the host does not know
// how many there are.
template <class U>
__global__ __launch_bounds__(kCopyThreads) void k_compact_move(Cache c, const int32_t* ws,
                                                               const int32_t* to,
                                                               const int32_t* from,
                                                               int64_t pieces, int piece_units) {
  const int moves = ws[0];
  if (moves == 0) return;
  const int first = from[0];
  for (int row = blockIdx.x; row < c.R; row += gridDim.x) {
    const int64_t len = c.lens[row];
    if (!len_ok(c, len)) continue;
    const int nblk = blocks_of(c, len);
    for (int b = threadIdx.x; b < nblk; b += kCopyThreads) {
      const int p = entry(c, row, b);
      if (p < first) continue;
      const int j = last_at_most(from, moves, p);
      if (from[j] == p) entry(c, row, b) = to[j];
    }
  }
  const uint32_t units = (uint32_t)((int64_t)c.P * c.C * 2 / sizeof(U));
  for (int64_t w = blockIdx.x; w < moves * pieces; w += gridDim.x) {
    const int j = (int)quotient(w, pieces);
    copy_piece<U>(c, from[j], to[j], units, w - j * pieces, piece_units);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
Cache view(const cg_paged_cache& c) {
  return {c.layers, c.channels, c.page_tokens, __builtin_ctz((unsigned)c.page_tokens),
          c.num_pages, c.n_rows, c.max_blocks, (char*)c.k_pool_dev, (char*)c.v_pool_dev,
          c.tables_dev, c.lens_dev, c.refs_dev, c.status_dev};
}

// The widest unit that every address and size is a multiple of: 16 bytes in any
// model's shape, 4 or 2 for odd channel counts or views of a buffer.
int unit_of(uint64_t bits) { return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2; }
uint64_t pool_bits(const cg_paged_cache& c) { return (uintptr_t)c.k_pool_dev | (uintptr_t)c.v_pool_dev; }

#define BY_UNIT(unit, call)                        \
  do {                                             \
    if ((unit) == 16) { using U = u32x4; call; }   \
    else if ((unit) == 4) { using U = uint32_t; call; } \
    else { using U = uint16_t; call; }             \
  } while (0)

int piece_for(int64_t copies, int L, int64_t units) {
  return copies * 2 * L * units >= (int64_t)2048 * kPieceMost ? kPieceMost : kPieceLeast;
}

int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? CG_OK : hip_fail(e, what);
}

int check_workspace(const cg_paged_cache* c, const void* ws, size_t bytes) {
  if (!ws || (uintptr_t)ws % 16) return fail(CG_E_INVAL, "workspace NULL or not 16-byte aligned");
  if (bytes < 4 * pages_ws(*c).words) return fail(CG_E_CAPACITY, "workspace too small");
  return CG_OK;
}

constexpr int64_t kMaxGrid = 1 << 20;

}  // namespace
}  // namespace cg

using namespace cg;

extern "C" {

int cg_pages_workspace(const cg_paged_cache* c, size_t* bytes) {
  if (int rc = check_paged_cache(c)) return rc;
  if (!bytes) return fail(CG_E_INVAL, "bytes is NULL");
  *bytes = 4 * pages_ws(*c).words;
  return CG_OK;
}

int cg_pages_copy_async(const cg_paged_cache* c, int32_t n, const int32_t* src_dev,
                        const int32_t* dst_dev, void* stream) {
  if (int rc = check_paged_cache(c)) return rc;
  if (n < 0 || n > c->num_pages) return fail(CG_E_INVAL, "n must be in 0..num_pages");
  if (n == 0) return CG_OK;
  if (!src_dev || !dst_dev) return fail(CG_E_INVAL, "NULL list");
  DeviceGuard dg(c->device);
  if (!dg.ok) return fail(CG_E_HIP, "cannot select the cache's device");
  const int64_t page = (int64_t)c->page_tokens * c->channels * 2;
  const int unit = unit_of((uint64_t)page | pool_bits(*c));
  const int piece = piece_for(n, c->layers, page / unit);
  const int64_t pieces = pieces_of(c->layers, page / unit, piece);
  if (n <= kFewPairs) {
    const int grid = (int)std::min(n * pieces, kMaxGrid);
    BY_UNIT(unit, (k_pages_copy<U><<<grid, kCopyThreads, 0, (hipStream_t)stream>>>(
                      view(*c), n, src_dev, dst_dev, pieces, piece)));
  } else {
    const int run = (n + kRuns - 1) / kRuns;
    BY_UNIT(unit, (k_pages_copy_many<U><<<(n + run - 1) / run, kRunThreads, 0, (hipStream_t)stream>>>(
                      view(*c), n, src_dev, dst_dev, run, pieces, piece)));
  }
  return launched("page copy");
}

int cg_pages_reserve_async(const cg_paged_cache* c, int32_t n, const int32_t* rows_dev,
                           const int32_t* starts_dev, int32_t n_tokens, int64_t* slots_dev,
                           void* workspace_dev, size_t workspace_bytes, void* stream) {
  if (int rc = check_paged_cache(c)) return rc;
  if (n < 0 || n > c->n_rows || n_tokens < 0 || n_tokens > kMaxTokens)
    return fail(CG_E_INVAL, "n must be in 0..n_rows and n_tokens in 0..2^21");
  if (n == 0 && (n_tokens == 0 || !slots_dev)) return CG_OK;
  if (n > 0 && (!rows_dev || !starts_dev)) return fail(CG_E_INVAL, "NULL list");
  if (int rc = check_workspace(c, workspace_dev, workspace_bytes)) return rc;
  DeviceGuard dg(c->device);
  if (!dg.ok) return fail(CG_E_HIP, "cannot select the cache's device");
  const PagesWs w = pages_ws(*c);
  int32_t* ws = (int32_t*)workspace_dev;
  if (n > 0 && n <= kFew)  // without a request there is no list to read the first one from
    k_reserve_few<<<1, kThreads, 0, (hipStream_t)stream>>>(view(*c), n, rows_dev, starts_dev,
                                                           n_tokens, slots_dev, ws + w.list);
  else
    k_reserve<<<1, kThreads, 0, (hipStream_t)stream>>>(view(*c), n, rows_dev, starts_dev, n_tokens,
                                                       slots_dev, ws + w.cum, ws + w.ok, ws + w.list);
  return launched("reserve");
}

int cg_pages_write_async(const cg_paged_cache* c, int32_t layer0, int32_t n_layers,
                         int32_t n_tokens, const int64_t* slots_dev, const void* k_new_dev,
                         const void* v_new_dev, int64_t token_stride, int64_t layer_stride,
                         void* stream) {
  if (int rc = check_paged_cache(c)) return rc;
  if (layer0 < 0 || n_layers < 0 || layer0 > c->layers - n_layers)
    return fail(CG_E_INVAL, "layers out of range");
  if (n_tokens < 0 || n_tokens > kMaxTokens)
    return fail(CG_E_INVAL, "n_tokens must be in 0..2^21");
  const int64_t most = (int64_t)1 << 40;
  if (token_stride < c->channels || token_stride > most || layer_stride < 0 || layer_stride > most)
    return fail(CG_E_INVAL, "token_stride must be at least channels, layer_stride not negative");
  if (n_layers == 0 || n_tokens == 0) return CG_OK;
  if (!slots_dev || !k_new_dev || !v_new_dev) return fail(CG_E_INVAL, "NULL argument");
  DeviceGuard dg(c->device);
  if (!dg.ok) return fail(CG_E_HIP, "cannot select the cache's device");
  const int64_t row = (int64_t)c->channels * 2;
  const int unit = unit_of((uint64_t)row | pool_bits(*c) | (uintptr_t)k_new_dev |
                           (uintptr_t)v_new_dev | (uint64_t)(2 * token_stride) |
                           (uint64_t)(n_layers > 1 ? 2 * layer_stride : 0));
  const uint32_t units = (uint32_t)(row / unit);
  const int piece = piece_for(n_tokens, n_layers, units);
  const int tile = (int)std::max<int64_t>(1, piece / units);
  const dim3 grid((unsigned)((n_tokens + tile - 1) / tile), 2 * n_layers);
  BY_UNIT(unit, (k_write<U><<<grid, kCopyThreads, 0, (hipStream_t)stream>>>(
                    view(*c), layer0, n_layers, n_tokens, slots_dev, (const char*)k_new_dev,
                    (const char*)v_new_dev, 2 * token_stride, 2 * layer_stride, units, tile)));
  return launched("page write");
}

int cg_pages_fork_async(const cg_paged_cache* c, int32_t n, const int32_t* parents_dev,
                        const int32_t* children_dev, void* workspace_dev, size_t workspace_bytes,
                        void* stream) {
  if (int rc = check_paged_cache(c)) return rc;
  if (n < 0 || n > c->n_rows) return fail(CG_E_INVAL, "n must be in 0..n_rows");
  if (n == 0) return CG_OK;
  if (!parents_dev || !children_dev) return fail(CG_E_INVAL, "NULL list");
  if (int rc = check_workspace(c, workspace_dev, workspace_bytes)) return rc;
  DeviceGuard dg(c->device);
  if (!dg.ok) return fail(CG_E_HIP, "cannot select the cache's device");
  const PagesWs w = pages_ws(*c);
  int32_t* ws = (int32_t*)workspace_dev;
  hipStream_t st = (hipStream_t)stream;
  if (n <= kFew)
    k_fork_plan_few<<<1, kThreads, 0, st>>>(view(*c), n, parents_dev, children_dev, ws + w.ok,
                                            ws + w.aux);
  else
    k_fork_plan<<<1, kThreads, 0, st>>>(view(*c), n, parents_dev, children_dev, ws + w.ok,
                                        ws + w.cum, ws + w.aux, ws + w.list);
  if (int rc = launched("fork")) return rc;
  // the copy's rows are known on the device only: pieces for a full page, the
  // surplus workgroups return at once
  const int64_t row = (int64_t)c->channels * 2;
  const int unit = unit_of((uint64_t)row | pool_bits(*c));
  const int piece = piece_for(n, c->layers, (c->page_tokens - 1) * row / unit);
  const int64_t pieces = pieces_of(c->layers, (c->page_tokens - 1) * row / unit, piece);
  const dim3 grid(n, (unsigned)(1 + std::min<int64_t>(pieces, std::max<int64_t>(1, 32768 / n))));
  BY_UNIT(unit, (k_fork_copy<U><<<grid, kCopyThreads, 0, st>>>(view(*c), parents_dev, children_dev,
                                                               ws + w.ok, ws + w.aux, piece)));
  return launched("fork");
}

int cg_pages_free_async(const cg_paged_cache* c, int32_t n, const int32_t* rows_dev,
                        void* stream) {
  if (int rc = check_paged_cache(c)) return rc;
  if (n < 0 || n > c->n_rows) return fail(CG_E_INVAL, "n must be in 0..n_rows");
  if (n == 0) return CG_OK;
  if (!rows_dev) return fail(CG_E_INVAL, "NULL list");
  DeviceGuard dg(c->device);
  if (!dg.ok) return fail(CG_E_HIP, "cannot select the cache's device");
  k_free<<<n, kCopyThreads, 0, (hipStream_t)stream>>>(view(*c), n, rows_dev);
  return launched("free");
}

int cg_pages_compact_async(const cg_paged_cache* c, int32_t* n_live_dev, void* workspace_dev,
                           size_t workspace_bytes, void* stream) {
  if (int rc = check_paged_cache(c)) return rc;
  if (int rc = check_workspace(c, workspace_dev, workspace_bytes)) return rc;
  DeviceGuard dg(c->device);
  if (!dg.ok) return fail(CG_E_HIP, "cannot select the cache's device");
  const PagesWs w = pages_ws(*c);
  int32_t* ws = (int32_t*)workspace_dev;
  hipStream_t st = (hipStream_t)stream;
  if (c->num_pages <= kScanPages)
    k_compact_plan_few<<<1, kThreads, 0, st>>>(view(*c), n_live_dev, ws, ws + w.list, ws + w.list2);
  else
    k_compact_plan<<<1, kThreads, 0, st>>>(view(*c), n_live_dev, ws, ws + w.list, ws + w.list2);
  if (int rc = launched("compact")) return rc;
  const int64_t page = (int64_t)c->page_tokens * c->channels * 2;
  const int unit = unit_of((uint64_t)page | pool_bits(*c));
  const int piece = piece_for(c->num_pages / 4, c->layers, page / unit);
  const int64_t pieces = pieces_of(c->layers, page / unit, piece);
  const int grid = (int)std::min<int64_t>(2048, std::max<int64_t>(c->n_rows, c->num_pages / 2 * pieces));
  BY_UNIT(unit, (k_compact_move<U><<<grid, kCopyThreads, 0, st>>>(view(*c), ws, ws + w.list,
                                                                  ws + w.list2, pieces, piece)));
  return launched("compact");
}

}  // extern "C"
