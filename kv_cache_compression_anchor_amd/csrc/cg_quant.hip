// Caches held in 4 bits: writing tokens and reading them back (include/cachegen.h,
// "Caches held in 4 bits").
//
// A thread takes 8 channels, 16 bytes of binary16 and one 32-bit word of codes; the four
// threads of a quad share a group's scale.  Decisions next to a border are exact in
// binary32: with 11 bits of x and 8 of s, x / s is a half or at least 2^-12 off one, and
// a / 7 is a number of 8 bits or at least 2^-12 of itself off one, so that a margin well
// below these and well above binary32's errors replaces exact quotients.
//
// What bounds it: memory.  4,666 tokens of 32 layers and 1,024 channels with the held numbers (1.40 GB)
// are written in 290 us, 4.8 TB/s (a copy reaches 4.9); 9,216 tokens of them are read back in 270
// us, 5.7 TB/s, as most of it is written.  A step's tokens of 64 requests (19 MB) take 6.8 us, four
// tokens of a small model 2.3.
#include <algorithm>

#include "cg_hostapi.h"
#include "cg_internal.h"
#include "cg_paged.h"

namespace cg {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kPer = 4;  // words of a thread: their loads are issued together
constexpr uint32_t kBadPage = 2u;  // status bit

struct Quant {
  int P, N, kv, d;
  int units;  // words of codes of a row
  int words, scales, row;  // of a head, where the scales begin, bytes of the row
  char *k, *v;
  uint32_t* status;
};

// 8 channels of one head from memory whose alignment is U's, or zeros behind the head.
template <class U>
__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
  union { u32x4 x; U u[16 / sizeof(U)]; } y;
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(U)); i++) y.u[i] = ((const U*)p)[i];
  return y.x;
}
template <class U>
__device__ __forceinline__ void store8(uint16_t* p, u32x4 x) {
  union { u32x4 x; U u[16 / sizeof(U)]; } y;
  y.x = x;
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(U)); i++) ((U*)p)[i] = y.u[i];
}

__device__ __forceinline__ uint32_t max_u16(uint32_t a, uint32_t b) {
  typedef uint16_t us2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, a), __builtin_bit_cast(us2, b)));
}

// Bits of the largest magnitude among the quad's 32 channels: binary16 magnitudes are
// ordered as whole numbers, infinities and NaNs above all others.
__device__ __forceinline__ uint32_t peak(u32x4 x) {
  uint32_t m = max_u16(max_u16(x[0] & 0x7FFF7FFFu, x[1] & 0x7FFF7FFFu), max_u16(x[2] & 0x7FFF7FFFu, x[3] & 0x7FFF7FFFu));
  m = max_u16(m, m >> 16) & 0xFFFFu;
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));  // lane ^ 1
  return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));  // lane ^ 2
}

// The scale of a group whose largest magnitude is a (finite): a / 7 rounded up to 8
// significant bits, or to binary16's smallest step.
__device__ __forceinline__ float scale_of(float a) {
  const float q = a * (float)((1 - 0x1p-20) / 7);  // less than a / 7, by less than what decides
  const float up = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, q) + 0xFFFFu) & 0xFFFF0000u);
  return fminf(q < 0x1p-16f ? ceilf(q * 0x1p24f) * 0x1p-24f : up, 9344.0f);
}

// 8 channels to their codes; held: the numbers that the codes stand for.
__device__ __forceinline__ uint32_t encode8(u32x4 x, float s, bool finite, u32x4& held) {
  const float inv = s == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(s);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    float y[2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const float v = half_bits_to_float((uint16_t)(x[i] >> 16 * j));
      const uint32_t n = (uint32_t)__builtin_fmaf(v, inv, (float)(8.5 + 0x1p-14));
      word |= n << (16 * j + 4 * i);
      y[j] = ((float)n - 8.0f) * s;
    }
    held[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)y[0]) |
              (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)y[1]) << 16;
  }
  if (!finite) {
    word = 0x88888888u;
    held = u32x4{0x7E007E00u, 0x7E007E00u, 0x7E007E00u, 0x7E007E00u};
  }
  return word;
}

struct Tensors {  // of new, held or read tokens
  const char *k, *v;
  int64_t token, layer;  // strides in bytes
};

// A workgroup takes `tile` tokens of one (kv, layer); the words of a row are numbered
// through.  kWhole: heads of whole groups, so that a row's channels are its words' too.
template <class U, bool kWhole, bool kHeld>
__global__ __launch_bounds__(kThreads) void k_quant_write(Quant c, int layer0, int n_layers, int n_tokens,
                                                          const int64_t* slots, Tensors in, Tensors held, int tile) {
  const int sl = blockIdx.y, l = sl < n_layers ? sl : sl - n_layers;
  const bool second = sl >= n_layers;
  const char* from = (second ? in.v : in.k) + l * in.layer;
  char* back = (char*)(second ? held.v : held.k) + l * held.layer;
  char* to = (second ? c.v : c.k) + (int64_t)(layer0 + l) * c.N * c.P * c.row;
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  const uint32_t nt = (uint32_t)(n_tokens - t0 < tile ? n_tokens - t0 : tile);
  const int64_t cap = (int64_t)c.N * c.P;
  const uint32_t all = nt * c.units;  // a multiple of 4: a quad is in it or not
  for (uint32_t e0 = threadIdx.x; e0 < all; e0 += kPer * kThreads) {
    u32x4 x[kPer];
    int64_t slot[kPer];
    uint32_t tok[kPer], unit[kPer], ch[kPer];
    bool in_head[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const uint32_t e = min(e0 + i * kThreads, all - 4 + (threadIdx.x & 3));
      tok[i] = e / c.units;
      unit[i] = e - tok[i] * c.units;
      const uint32_t head = kWhole ? 0 : unit[i] / c.words, w = unit[i] - head * c.words;
      ch[i] = head * c.d + w * 8;
      in_head[i] = kWhole || w * 8 < (uint32_t)c.d;
      x[i] = u32x4{0, 0, 0, 0};
      if (in_head[i]) x[i] = load8<U>((const uint16_t*)(from + (t0 + tok[i]) * in.token) + ch[i]);
      slot[i] = slots[t0 + tok[i]];
    }
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      if (e0 + i * kThreads >= all) break;
      const uint32_t bits = peak(x[i]);
      const bool finite = bits < 0x7C00u;
      const float s = scale_of(half_bits_to_float((uint16_t)bits));
      u32x4 y;
      const uint32_t word = encode8(x[i], s, finite, y);
      if (kHeld && in_head[i]) store8<U>((uint16_t*)(back + (t0 + tok[i]) * held.token) + ch[i], y);
      if (slot[i] >= 0 && slot[i] < cap) {
        char* row = to + slot[i] * c.row;
        ((uint32_t*)row)[unit[i]] = word;
        if (unit[i] % 4 == 0)
          ((uint16_t*)(row + c.scales))[unit[i] / 4] =
              finite ? __builtin_bit_cast(uint16_t, (_Float16)s) : (uint16_t)0x7E00u;
      } else if (slot[i] != -1 && unit[i] == 0) {
        atomicOr(c.status, kBadPage);
      }
    }
  }
}

template <class U, bool kWhole>
__global__ __launch_bounds__(kThreads) void k_quant_read(Quant c, int layer0, int n_layers, int n_tokens,
                                                         const int64_t* slots, Tensors out, int tile) {
  const int sl = blockIdx.y, l = sl < n_layers ? sl : sl - n_layers;
  const bool second = sl >= n_layers;
  char* to = (char*)(second ? out.v : out.k) + l * out.layer;
  const char* from = (second ? c.v : c.k) + (int64_t)(layer0 + l) * c.N * c.P * c.row;
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  const uint32_t nt = (uint32_t)(n_tokens - t0 < tile ? n_tokens - t0 : tile);
  const int64_t cap = (int64_t)c.N * c.P;
  const uint32_t all = nt * c.units;
  for (uint32_t e0 = threadIdx.x; e0 < all; e0 += kPer * kThreads) {
    int64_t slot[kPer];
    uint32_t tok[kPer], unit[kPer], word[kPer];
    uint16_t scale[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const uint32_t e = min(e0 + i * kThreads, all - 1);
      tok[i] = e / c.units;
      unit[i] = e - tok[i] * c.units;
      slot[i] = slots[t0 + tok[i]];
    }
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const char* row = from + (slot[i] >= 0 && slot[i] < cap ? slot[i] : 0) * c.row;
      word[i] = ((const uint32_t*)row)[unit[i]];
      scale[i] = ((const uint16_t*)(row + c.scales))[unit[i] / 4];
    }
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      if (e0 + i * kThreads >= all) break;
      if (slot[i] < 0 || slot[i] >= cap) {
        if (slot[i] != -1 && unit[i] == 0) atomicOr(c.status, kBadPage);
        continue;
      }
      const uint32_t head = kWhole ? 0 : unit[i] / c.words, w = unit[i] - head * c.words;
      if (!kWhole && w * 8 >= (uint32_t)c.d) continue;
      const float s = half_bits_to_float(scale[i]);
      u32x4 y;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float a = (float)(int)((word[i] >> 4 * j & 15) - 8) * s, b = (float)(int)((word[i] >> (16 + 4 * j) & 15) - 8) * s;
        y[j] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) |
               (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16;
      }
      store8<U>((uint16_t*)(to + (t0 + tok[i]) * out.token) + head * c.d + w * 8, y);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
Quant view(const cg_paged_cache& c, const cg_quant_form& f) {
  const QuantRow r = quant_row(f);
  return {c.page_tokens, c.num_pages, f.channels / f.head_dim, f.head_dim, r.scales / 4, r.head / 4, r.scales, r.row,
          (char*)c.k_pool_dev, (char*)c.v_pool_dev, c.status_dev};
}

// Checks that writing and reading share.
int check(const cg_paged_cache* c, const cg_quant_form* f, int layer0, int n_layers, int n_tokens, int64_t token_stride,
          int64_t layer_stride) {
  if (int rc = check_quant(c, f)) return rc;
  if (layer0 < 0 || n_layers < 0 || layer0 > c->layers - n_layers)
    return fail(CG_E_INVAL, "layers out of range");
  if (n_tokens < 0 || n_tokens > kMaxTokens)
    return fail(CG_E_INVAL, "n_tokens must be in 0..2^21");
  const int64_t most = (int64_t)1 << 40;
  if (token_stride < f->channels || token_stride > most || layer_stride < 0 || layer_stride > most)
    return fail(CG_E_INVAL, "token_stride must be at least channels, layer_stride not negative");
  return CG_OK;
}

// The widest unit of 16, 4 or 2 bytes that a tensor's addresses are multiples of (heads begin
// at multiples of 16 bytes).
int unit_of(uint64_t bits) { return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2; }
uint64_t bits_of(const void* k, const void* v, int64_t token, int64_t layer, int n_layers) {
  return (uintptr_t)k | (uintptr_t)v | (uint64_t)(2 * token) | (uint64_t)(n_layers > 1 ? 2 * layer : 0);
}

// Tokens of a workgroup: kPer words a thread where there is enough to do, one where
// workgroups are scarce.
int tile_for(int64_t n_tokens, int n_layers, int units) {
  const bool many = n_tokens * 2 * n_layers * units >= (int64_t)2048 * kPer * kThreads;
  return std::max(1, (many ? kPer * kThreads : kThreads) / units);
}

int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? CG_OK : hip_fail(e, what);
}

template <class U>
void write(const Quant& q, int layer0, int n_layers, int n_tokens, const int64_t* slots, const Tensors& in,
           const Tensors& held, hipStream_t st) {
  const int tile = tile_for(n_tokens, n_layers, q.units);
  const dim3 grid((unsigned)((n_tokens + tile - 1) / tile), 2 * n_layers);
#define GO(WHOLE, HELD)                                                                                             \
  if ((q.d % 32 == 0) == WHOLE && (held.k != nullptr) == HELD)                                                      \
    k_quant_write<U, WHOLE, HELD><<<grid, kThreads, 0, st>>>(q, layer0, n_layers, n_tokens, slots, in, held, tile);
  GO(true, true) GO(true, false) GO(false, true) GO(false, false)
#undef GO
}
template <class U>
void read(const Quant& q, int layer0, int n_layers, int n_tokens, const int64_t* slots, const Tensors& out,
          hipStream_t st) {
  const int tile = tile_for(n_tokens, n_layers, q.units);
  const dim3 grid((unsigned)((n_tokens + tile - 1) / tile), 2 * n_layers);
  if (q.d % 32 == 0) k_quant_read<U, true><<<grid, kThreads, 0, st>>>(q, layer0, n_layers, n_tokens, slots, out, tile);
  else k_quant_read<U, false><<<grid, kThreads, 0, st>>>(q, layer0, n_layers, n_tokens, slots, out, tile);
}

}  // namespace
}  // namespace cg

using namespace cg;

extern "C" {

int cg_quant_write_async(const cg_paged_cache* c, const cg_quant_form* f, int32_t layer0, int32_t n_layers,
                         int32_t n_tokens, const int64_t* slots_dev, const void* k_new_dev, const void* v_new_dev,
                         int64_t token_stride, int64_t layer_stride, void* k_held_dev, void* v_held_dev,
                         int64_t held_token_stride, int64_t held_layer_stride, void* stream) {
  if (int rc = check(c, f, layer0, n_layers, n_tokens, token_stride, layer_stride)) return rc;
  if (!k_held_dev != !v_held_dev) return fail(CG_E_INVAL, "k_held and v_held must both be given or neither");
  if (k_held_dev)
    if (int rc = check(c, f, layer0, n_layers, n_tokens, held_token_stride, held_layer_stride)) return rc;
  if (n_layers == 0 || n_tokens == 0) return CG_OK;
  if (!slots_dev || !k_new_dev || !v_new_dev) return fail(CG_E_INVAL, "NULL argument");
  DeviceGuard dg(c->device);
  if (!dg.ok) return fail(CG_E_HIP, "cannot select the cache's device");
  const Quant q = view(*c, *f);
  const Tensors in{(const char*)k_new_dev, (const char*)v_new_dev, 2 * token_stride, 2 * layer_stride};
  const Tensors held{(const char*)k_held_dev, (const char*)v_held_dev, 2 * held_token_stride, 2 * held_layer_stride};
  uint64_t bits = bits_of(k_new_dev, v_new_dev, token_stride, layer_stride, n_layers);
  if (k_held_dev) bits |= bits_of(k_held_dev, v_held_dev, held_token_stride, held_layer_stride, n_layers);
  const int unit = unit_of(bits);
  hipStream_t st = (hipStream_t)stream;
  if (unit == 16) write<u32x4>(q, layer0, n_layers, n_tokens, slots_dev, in, held, st);
  else if (unit == 4) write<uint32_t>(q, layer0, n_layers, n_tokens, slots_dev, in, held, st);
  else write<uint16_t>(q, layer0, n_layers, n_tokens, slots_dev, in, held, st);
  return launched("write in 4 bits");
}

int cg_quant_read_async(const cg_paged_cache* c, const cg_quant_form* f, int32_t layer0, int32_t n_layers,
                        int32_t n_tokens, const int64_t* slots_dev, void* k_out_dev, void* v_out_dev,
                        int64_t token_stride, int64_t layer_stride, void* stream) {
  if (int rc = check(c, f, layer0, n_layers, n_tokens, token_stride, layer_stride)) return rc;
  if (n_layers == 0 || n_tokens == 0) return CG_OK;
  if (!slots_dev || !k_out_dev || !v_out_dev) return fail(CG_E_INVAL, "NULL argument");
  DeviceGuard dg(c->device);
  if (!dg.ok) return fail(CG_E_HIP, "cannot select the cache's device");
  const Quant q = view(*c, *f);
  const Tensors out{(const char*)k_out_dev, (const char*)v_out_dev, 2 * token_stride, 2 * layer_stride};
  const int unit = unit_of(bits_of(k_out_dev, v_out_dev, token_stride, layer_stride, n_layers));
  hipStream_t st = (hipStream_t)stream;
  if (unit == 16) read<u32x4>(q, layer0, n_layers, n_tokens, slots_dev, out, st);
  else if (unit == 4) read<uint32_t>(q, layer0, n_layers, n_tokens, slots_dev, out, st);
  else read<uint16_t>(q, layer0, n_layers, n_tokens, slots_dev, out, st);
  return launched("read of 4 bits");
}

}  // extern "C"
