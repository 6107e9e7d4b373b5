// Prints how calls of the attention over caches held in 4 bits are launched (csrc/cg_quant_plan.h).  Each
// line of the input: channels, head_dim, page_tokens, max_blocks, n_heads, n_seqs, n_q, n_groups,
// max_q, max_prefix, max_len.  Each of the output: channels of a head that the kernel takes, how a
// prefix's and how the rest's rows are held, how the tokens are cut, and into how many splits or parts.
#include <cstdio>

#include "cg_quant_plan.h"

int main() {
  cg_quant_form f{};
  cg_paged_cache c{};
  cg_attention x{};
  while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d", &f.channels, &f.head_dim, &c.page_tokens, &c.max_blocks, &x.n_heads,
                    &x.n_seqs, &x.n_q, &x.n_groups, &x.max_q, &x.max_prefix, &x.max_len) == 11) {
    x.head_dim = f.head_dim;
    c.channels = cg::quant_row(f).row / 2;
    const cg::Plan p = cg::plan_of(c, f, x);
    std::printf("%d %d %d %d %d\n", p.dp, p.pre_mode, p.rest_mode, p.cut(), p.parts ? p.parts : p.rest_splits);
  }
}
