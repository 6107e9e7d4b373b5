// Host-side checks of the paged-cache calls' numbers and pointers.  No HIP here.
#include <math.h>

#include "cg_paged.h"

namespace cg {

int check_paged_cache(const cg_paged_cache* c) {
  if (!c) return fail(CG_E_INVAL, "cache is NULL");
  if (c->device < 0) return fail(CG_E_INVAL, "device must not be negative");
  if (c->layers < 1 || c->layers > 4096 || c->channels < 1 || c->channels > 65536)
    return fail(CG_E_INVAL, "layers must be in 1..4096 and channels in 1..65536");
  if (c->page_tokens < 1 || c->page_tokens > kMaxChunk || (c->page_tokens & (c->page_tokens - 1)))
    return fail(CG_E_INVAL, "page_tokens must be a power of two in [1, 65536]");
  if ((uint64_t)c->page_tokens * (uint64_t)c->channels * 2u >= (1ull << 32))
    return fail(CG_E_INVAL, "a page of one layer must be smaller than 4 GiB");
  if (c->num_pages < 1 || c->num_pages > 1 << 24)
    return fail(CG_E_INVAL, "num_pages must be in 1..2^24");
  if (c->n_rows < 1 || c->n_rows > 65536) return fail(CG_E_INVAL, "n_rows must be in 1..65536");
  if (c->max_blocks < 1 || (int64_t)c->max_blocks * c->page_tokens > (int64_t)1 << 30)
    return fail(CG_E_INVAL, "max_blocks must be positive and max_blocks x page_tokens at most 2^30");
  if (c->reserved != 0) return fail(CG_E_INVAL, "reserved must be 0");
  if (!c->k_pool_dev || !c->v_pool_dev || !c->tables_dev || !c->lens_dev || !c->refs_dev ||
      !c->status_dev)
    return fail(CG_E_INVAL, "NULL pointer in the cache");
  return CG_OK;
}

// The call's numbers on a cache of `channels` channels a token.
static int check_call(const cg_paged_cache* c, const cg_attention* a, int channels) {
  if (!a) return fail(CG_E_INVAL, "call is NULL");
  if (a->layer < 0 || a->layer >= c->layers) return fail(CG_E_INVAL, "layer out of range");
  if (a->head_dim < 8 || a->head_dim > 256 || a->head_dim % 8 || channels % a->head_dim)
    return fail(CG_E_INVAL, "head_dim must be a multiple of 8 up to 256 that divides channels");
  const int kv = channels / a->head_dim;
  if (a->n_heads < 1 || a->n_heads > 1024 || a->n_heads % kv)
    return fail(CG_E_INVAL, "n_heads must be a multiple of channels / head_dim, at most 1024");
  // scores are computed in units of log 2: the scale has to stay finite in them
  if (!(fabsf(a->scale) <= 0x1p127f)) return fail(CG_E_INVAL, "scale must be a number of at most 2^127 in size");
  if (a->n_seqs < 0 || a->n_seqs > c->n_rows || a->n_q < 0 || a->n_q > 1 << 20 ||
      a->n_groups < 0 || a->n_groups > a->n_seqs)
    return fail(CG_E_INVAL, "n_seqs, n_q or n_groups out of range");
  if (a->max_q < 0 || a->max_prefix < 0 || a->max_len < 0)
    return fail(CG_E_INVAL, "max_q, max_prefix and max_len must not be negative");
  return CG_OK;
}

int check_attention(const cg_paged_cache* c, const cg_attention* a) {
  if (int rc = check_paged_cache(c)) return rc;
  return check_call(c, a, c->channels);
}

int check_attention_strides(const cg_attention* a) {
  if (a->q_stride < (int64_t)a->n_heads * a->head_dim || a->q_stride > (int64_t)1 << 40 ||
      a->out_stride < (int64_t)a->n_heads * a->head_dim || a->out_stride > (int64_t)1 << 40 ||
      (a->q_stride | a->out_stride) % 8)
    return fail(CG_E_INVAL, "q_stride and out_stride must be multiples of 8 and at least n_heads x head_dim");
  return CG_OK;
}

int check_attention_memory(const cg_paged_cache* c, const cg_attention* a, const void* workspace,
                           size_t bytes, size_t need) {
  if (!a->q_starts_dev || !a->q_dev || !a->out_dev ||
      (a->n_groups > 0 && (!a->group_starts_dev || !a->prefix_lens_dev)))
    return fail(CG_E_INVAL, "NULL pointer in the call");
  if (((uintptr_t)a->q_dev | (uintptr_t)a->out_dev | (uintptr_t)c->k_pool_dev |
       (uintptr_t)c->v_pool_dev) % 16)
    return fail(CG_E_INVAL, "pools, q and out must be 16-byte aligned");
  if (!workspace || (uintptr_t)workspace % 16)
    return fail(CG_E_INVAL, "workspace NULL or not 16-byte aligned");
  if (bytes < need) return fail(CG_E_CAPACITY, "workspace too small");
  return CG_OK;
}

static int check_form(const cg_quant_form* f) {
  if (!f) return fail(CG_E_INVAL, "form is NULL");
  if (f->bits != 4 || f->reserved != 0) return fail(CG_E_INVAL, "bits must be 4 and reserved 0");
  if (f->channels < 1 || f->channels > 65536) return fail(CG_E_INVAL, "channels must be in 1..65536");
  if (f->head_dim < 8 || f->head_dim > 256 || f->head_dim % 8 || f->channels % f->head_dim)
    return fail(CG_E_INVAL, "head_dim must be a multiple of 8 up to 256 that divides channels");
  if (quant_row(*f).row > 2 * 65536) return fail(CG_E_INVAL, "a row would take more than 131,072 bytes");
  return CG_OK;
}

int check_quant(const cg_paged_cache* c, const cg_quant_form* f) {
  if (int rc = check_paged_cache(c)) return rc;
  if (int rc = check_form(f)) return rc;
  if (2 * c->channels != quant_row(*f).row)
    return fail(CG_E_INVAL, "the cache's channels are not those that cg_quant_row gives");
  if (((uintptr_t)c->k_pool_dev | (uintptr_t)c->v_pool_dev) % 16)
    return fail(CG_E_INVAL, "pools must be 16-byte aligned");
  return CG_OK;
}

int check_quant_attention(const cg_paged_cache* c, const cg_quant_form* f, const cg_attention* a) {
  if (int rc = check_quant(c, f)) return rc;
  if (int rc = check_call(c, a, f->channels)) return rc;
  if (a->head_dim != f->head_dim) return fail(CG_E_INVAL, "head_dim must be the form's");
  return CG_OK;
}

}  // namespace cg

extern "C" int cg_quant_row(const cg_quant_form* form, int32_t* cache_channels) {
  if (int rc = cg::check_form(form)) return rc;
  if (!cache_channels) return cg::fail(CG_E_INVAL, "cache_channels is NULL");
  *cache_channels = cg::quant_row(*form).row / 2;
  return CG_OK;
}
