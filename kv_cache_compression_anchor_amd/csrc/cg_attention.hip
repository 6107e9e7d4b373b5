// Attention of new tokens over a paged cache whose groups of sequences share a
// prefix (include/cachegen.h, cg_attention_prefix_async).
#include <algorithm>

#include "cg_hostapi.h"
#include "cg_internal.h"
#include "cg_paged.h"

namespace cg {
namespace {

constexpr uint32_t kBadPage = 2u, kRefused = 4u;  // status bits

struct Attn {
  int C, P, shift, N, R, B;
  const uint16_t *k, *v;  // the layer's pools
  const int32_t *tables, *lens;
  uint32_t* status;
  int H, G, d;  // query heads, heads per kv head, head dimension
  float scale;
  int n_seqs, n_q, n_groups;
  const int32_t *rows, *q_starts, *group_starts, *prefix_lens;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t q_stride, out_stride;
};

// largest i in [0, n) with a[i] <= x, or -1
__device__ __forceinline__ int last_at_most(const int32_t* a, int n, int x) {
  int lo = -1, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a[m] <= x) lo = m; else hi = m;
  }
  return lo;
}

struct Seq {
  bool ok;              // its row, length and prefix fit together
  int row, pre_row;     // rows of the tables that the rest and the prefix are read through
  int len, pre, q0, m;  // tokens, those of the prefix, first query, queries
};

__device__ __forceinline__ int row_of(const Attn& a, int s) { return a.rows ? a.rows[s] : s; }

__device__ __forceinline__ Seq sequence(const Attn& a, int s) {
  Seq q;
  q.row = row_of(a, s);
  q.q0 = a.q_starts[s];
  q.m = a.q_starts[s + 1] - q.q0;
  q.pre = 0;
  q.pre_row = q.row;
  const bool in = q.row >= 0 && q.row < a.R;
  q.len = in ? a.lens[q.row] : 0;
  q.ok = in && q.len >= 0 && q.len <= (int64_t)a.B << a.shift && q.q0 >= 0 &&
         a.q_starts[s + 1] <= a.n_q;
  if (a.n_groups) {
    const int g = last_at_most(a.group_starts, a.n_groups, s);
    if (g >= 0 && s < a.group_starts[g + 1]) {
      q.pre = a.prefix_lens[g];
      q.pre_row = row_of(a, a.group_starts[g] < 0 ? 0 : a.group_starts[g]);
      q.ok = q.ok && q.pre_row >= 0 && q.pre_row < a.R && q.pre >= 0 &&
             (q.pre == 0 || (int64_t)q.pre + q.m <= q.len);
    }
  }
  return q;
}

// One workgroup per (query token, head): 256 tokens at a time, a thread scores
// one token, then a thread sums one channel.
__global__ __launch_bounds__(256) void k_attention(Attn a) {
  __shared__ float qs[256], p[256], red[256];
  __shared__ int64_t at[256];
  const int qi = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, kvh = h / a.G;
  const int s = last_at_most(a.q_starts, a.n_seqs, qi);
  if (s < 0 || qi >= a.q_starts[s + 1]) return;
  const Seq q = sequence(a, s);
  if (tid < a.d)
    qs[tid] = half_bits_to_float(a.q[qi * a.q_stride + h * a.d + tid]) * a.scale;
  int lim = q.len - q.m + (qi - q.q0) + 1;
  if (!q.ok) {
    lim = 0;
    if (tid == 0) atomicOr(a.status, kRefused);
  }
  float m = -__builtin_inff(), l = 0.0f, o = 0.0f;
  for (int base = 0; base < lim; base += 256) {
    const int t = base + tid;
    float x = -__builtin_inff();
    int64_t where = -1;
    if (t < lim) {
      const int page = a.tables[(int64_t)(t < q.pre ? q.pre_row : q.row) * a.B + (t >> a.shift)];
      if (page >= 0 && page < a.N)
        where = (((int64_t)page << a.shift) + (t & (a.P - 1))) * a.C + kvh * a.d;
      else
        atomicOr(a.status, kBadPage);
    }
    __syncthreads();  // qs is written; p, at and red of the last step are read
    if (where >= 0) {
      x = 0.0f;
      for (int i = 0; i < a.d; i++) x += qs[i] * half_bits_to_float(a.k[where + i]);
    }
    red[tid] = x;
    at[tid] = where;
    for (int w = 128; w; w >>= 1) {
      __syncthreads();
      if (tid < w) red[tid] = fmaxf(red[tid], red[tid + w]);
    }
    __syncthreads();
    const float nm = fmaxf(m, red[0]);
    const float keep = nm == -__builtin_inff() ? 1.0f : __expf(m - nm);
    p[tid] = x == -__builtin_inff() ? 0.0f : __expf(x - nm);
    __syncthreads();
    l *= keep;
    o *= keep;
    m = nm;
    for (int i = 0; i < 256; i++) {
      l += p[i];
      if (tid < a.d && at[i] >= 0) o += p[i] * half_bits_to_float(a.v[at[i] + tid]);
    }
  }
  if (tid < a.d) a.out[qi * a.out_stride + h * a.d + tid] = float_to_half_bits(l == 0 ? 0.0f : o / l);
  if (tid == 0 && a.lse) a.lse[(int64_t)qi * a.H + h] = l == 0 ? -__builtin_inff() : m + __logf(l);
}

Attn view(const cg_paged_cache& c, const cg_attention& x) {
  Attn a;
  a.C = c.channels;
  a.P = c.page_tokens;
  a.shift = __builtin_ctz((unsigned)c.page_tokens);
  a.N = c.num_pages;
  a.R = c.n_rows;
  a.B = c.max_blocks;
  const int64_t layer = (int64_t)x.layer * c.num_pages * c.page_tokens * c.channels;
  a.k = (const uint16_t*)c.k_pool_dev + layer;
  a.v = (const uint16_t*)c.v_pool_dev + layer;
  a.tables = c.tables_dev;
  a.lens = c.lens_dev;
  a.status = c.status_dev;
  a.H = x.n_heads;
  a.d = x.head_dim;
  a.G = x.n_heads / (c.channels / x.head_dim);
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

using namespace cg;

extern "C" {

int cg_attention_workspace(const cg_paged_cache* c, const cg_attention* a, size_t* bytes) {
  if (int rc = check_attention(c, a)) return rc;
  if (!bytes) return fail(CG_E_INVAL, "bytes is NULL");
  *bytes = 16;
  return CG_OK;
}

int cg_attention_prefix_async(const cg_paged_cache* c, const cg_attention* a, void* workspace_dev,
                              size_t workspace_bytes, void* stream) {
  if (int rc = check_attention(c, a)) return rc;
  size_t need = 0;
  if (int rc = cg_attention_workspace(c, a, &need)) return rc;
  if (a->q_stride < (int64_t)a->n_heads * a->head_dim || a->q_stride > (int64_t)1 << 40 ||
      a->out_stride < (int64_t)a->n_heads * a->head_dim || a->out_stride > (int64_t)1 << 40 ||
      (a->q_stride | a->out_stride) % 8)
    return fail(CG_E_INVAL, "q_stride and out_stride must be multiples of 8 and at least n_heads x head_dim");
  if (a->n_seqs == 0 || a->n_q == 0) return CG_OK;
  if (!a->q_starts_dev || !a->q_dev || !a->out_dev ||
      (a->n_groups > 0 && (!a->group_starts_dev || !a->prefix_lens_dev)))
    return fail(CG_E_INVAL, "NULL pointer in the call");
  if (((uintptr_t)a->q_dev | (uintptr_t)a->out_dev | (uintptr_t)c->k_pool_dev |
       (uintptr_t)c->v_pool_dev) % 16)
    return fail(CG_E_INVAL, "pools, q and out must be 16-byte aligned");
  if (!workspace_dev || (uintptr_t)workspace_dev % 16)
    return fail(CG_E_INVAL, "workspace NULL or not 16-byte aligned");
  if (workspace_bytes < need) return fail(CG_E_CAPACITY, "workspace too small");
  DeviceGuard dg(c->device);
  if (!dg.ok) return fail(CG_E_HIP, "cannot select the cache's device");
  k_attention<<<dim3(a->n_q, a->n_heads), 256, 0, (hipStream_t)stream>>>(view(*c, *a));
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? CG_OK : hip_fail(e, "attention");
}

}  // extern "C"
