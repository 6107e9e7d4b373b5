// Paged-cache operators of libcachegen: the host-side checks of their arguments
// (plain C++, no HIP, so that they build on their own too) and the kernel
// launchers' arguments.
#pragma once

#include "cg_format.h"

namespace cg {

int check_paged_cache(const cg_paged_cache* c);
int check_attention(const cg_paged_cache* c, const cg_attention* a);

// Workspace of the page operators, in int32 words: [0] counters, then one
// entry per request (first page of request i in the dealt list, whether it was
// granted, three words of a fork's copy) and two per page (free pages dealt out,
// or the moves of a compaction and where a page went).
struct PagesWs {
  size_t cum, ok, aux, list, list2, words;
};
inline PagesWs pages_ws(const cg_paged_cache& c) {
  PagesWs w;
  size_t at = 16;
  w.cum = at;
  at += (size_t)c.n_rows + 4;
  w.ok = at;
  at += (size_t)c.n_rows;
  w.aux = at;
  at += (size_t)3 * c.n_rows;
  w.list = at;
  at += (size_t)c.num_pages;
  w.list2 = at;
  at += (size_t)c.num_pages;
  w.words = (at + 3) & ~(size_t)3;
  return w;
}

}  // namespace cg
