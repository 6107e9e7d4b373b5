// How calls of the attention over caches held in 4 bits are launched (csrc/cg_quant_plan.h), over
// random calls of the whole range: the kernel that a call asks for is one of those that are
// built, each of those is asked for by some call, and what the kernels take for granted of
// the launch's numbers holds.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "cg_quant_plan.h"

using namespace cg;

static void need(bool ok, const char* what) {
  if (!ok) {
    std::printf("%s\n", what);
    std::exit(1);
  }
}

int main() {
  std::mt19937_64 rng(7);
  auto upto = [&](int64_t n) { return (int64_t)(rng() % (uint64_t)(n + 1)); };
  auto spread = [&](int64_t n) {  // 0 .. n, as many of each order of magnitude
    const int bits = (int)upto(63 - __builtin_clzll((uint64_t)n | 1));
    return std::min(n, (int64_t)((2ull << bits) - 1) & (int64_t)rng());
  };
  int asked[3][kModes][kModes][kCuts] = {};
  const int dims[] = {8, 16, 32, 40, 64, 72, 80, 96, 128, 136, 160, 192, 200, 224, 248, 256};
  int calls = 0;
  for (int tries = 0; tries < 600000; tries++) {
    cg_quant_form f{};
    cg_paged_cache c{};
    cg_attention x{};
    const int d = dims[upto(15)], kv = 1 + (int)spread(255);
    f.head_dim = x.head_dim = d;
    f.channels = d * kv;
    if (f.channels > 65536) continue;
    const QuantRow r = quant_row(f);
    if (r.row > 2 * 65536) continue;
    c.channels = r.row / 2;
    c.page_tokens = 1 << upto(11);
    c.num_pages = 1 + (int)spread((1 << 24) - 1);
    c.n_rows = 1 + (int)spread(65535);
    c.max_blocks = 1 + (int)spread((1 << 30) / c.page_tokens - 1);
    x.n_heads = kv * (1 + (int)spread(1024 / kv - 1));
    x.n_seqs = (int)spread(c.n_rows);
    x.n_q = upto(3) ? (int)std::min<int64_t>(1 << 20, x.n_seqs * (1 + spread(600))) : (int)spread(1 << 20);
    x.n_groups = upto(2) ? (int)spread(x.n_seqs) : 0;
    x.max_q = upto(3) ? (int)spread(600) : (int)spread(INT32_MAX);
    x.max_prefix = upto(3) ? (int)spread(100000) : (int)spread(INT32_MAX);
    x.max_len = upto(3) ? (int)spread(200000) : (int)spread(INT32_MAX);
    const Plan p = plan_of(c, f, x);
    calls++;
    need(built(p.dp, p.pre_mode, p.rest_mode, p.cut()), "a call for a kernel that is not built");
    asked[p.dp / 128][p.pre_mode][p.rest_mode][p.cut()]++;
    need(d <= p.dp && p.rest_heads >= 1 && kv % p.rest_heads == 0 && p.pre_tiles >= 1 && p.rest_tiles >= 1 &&
             p.rest_splits >= 1 && p.rest_splits < 0x7FFF && p.pre_splits >= 0 && p.pre_splits < 0xFFFF &&
             p.pre_least >= 1 && p.rest_least >= 1,
         "numbers of the launch");
    need(!is_many(p.rest_mode) || p.rest_heads == 1, "many rows of several heads");
    need(p.direct || (kv % p.pre_heads == 0 && (is_many(p.pre_mode) ? p.pre_heads == 1 : p.pre_heads == p.rest_heads)),
         "heads of a prefix");
    need(p.direct ? p.pre_groups == 0 && p.pre_splits == 0 && p.rest_splits == 1 : p.pre_groups == x.n_groups, "groups");
    const int64_t columns = kv / p.rest_heads;
    const int64_t pre = (int64_t)p.pre_groups * p.pre_splits * p.pre_tiles * (kv / p.pre_heads);
    const int64_t items = pre + (p.parts ? p.parts : (int64_t)x.n_seqs * p.rest_splits) * p.rest_tiles * columns;
    need(items + (1 << 22) <= INT32_MAX, "an item's number passes 31 bits");
    if (p.parts) need(x.n_seqs <= kMostListed && items <= 1 << 22 && p.rest_splits >= 2, "parts");
    if (!p.direct)
      need(p.words >= (size_t)(p.pre_splits + p.rest_splits) * x.n_q * x.n_heads * (d + 2) + x.n_q, "room for the sums");
    if (!is_many(p.rest_mode)) {  // super tiles: a wave each for its head's tiles, in a stage of LDS
      const int waves = p.dp == 256 ? 4 : 8, n = p.rest_heads;
      need(p.turn >= 1 && p.turn * n <= waves, "tiles of a super tile");
      for (int head = 0; head < kv; head += n) {
        const int skew = (r.scales + 2 * head * r.groups) % 16, cpr = n * r.head / 16 + (skew + 2 * n * r.groups + 15) / 16;
        need(2 * ((p.turn * 512 * cpr + 1023) / 1024 * 1024) <= 37 * 1024, "a super tile does not fit");
      }
    }
  }
  need(calls > 100000, "too few calls");
  for (int dp : {64, 128, 256})
    for (int pre = 0; pre < kModes; pre++)
      for (int rest = 0; rest < kModes; rest++)
        for (int cut = 0; cut < kCuts; cut++)
          if (built(dp, pre, rest, cut) && !asked[dp / 128][pre][rest][cut]) {
            std::printf("no call asks for <%d, %d, %d, %d>\n", dp, pre, rest, cut);
            return 1;
          }
  std::printf("plans ok\n");
}
