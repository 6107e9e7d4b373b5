// Paged-cache operators of libcachegen: the host-side checks of their arguments
// (plain C++, no HIP, so that they build on their own too) and the kernel
// launchers' arguments.
#pragma once

#include "cg_format.h"

namespace cg {

int check_paged_cache(const cg_paged_cache* c);
int check_attention(const cg_paged_cache* c, const cg_attention* a);
int check_quant(const cg_paged_cache* c, const cg_quant_form* f);
int check_quant_attention(const cg_paged_cache* c, const cg_quant_form* f, const cg_attention* a);
// What a call and its workspace have to be like once its numbers are right.
int check_attention_strides(const cg_attention* a);
int check_attention_memory(const cg_paged_cache* c, const cg_attention* a, const void* workspace,
                           size_t bytes, size_t need);

// A row of a cache held in 4 bits, in bytes.
struct QuantRow {
  int head, groups;  // codes of a head, its groups of 32 channels
  int scales, row;   // where the scales begin, the whole row
};
inline QuantRow quant_row(const cg_quant_form& f) {
  QuantRow r;
  r.groups = (f.head_dim + 31) / 32;
  r.head = 16 * r.groups;
  const int heads = f.channels / f.head_dim;
  r.scales = heads * r.head;
  r.row = (r.scales + 2 * heads * r.groups + 15) & ~15;
  return r;
}

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
