// Shared parts of the quantised key-value cache: the views of the ABI's
// structs that the kernels take, the place of a token in the cache, the grid
// word and the element types.
#pragma once

#include "gptq_common.h"

namespace gptq {

// Keeps the compiler from seeing a constant, so that it stays in an SGPR or
// a VGPR instead of becoming a literal of every instruction that uses it.
// KV_FRESH_V makes a value new at every pass, so that nothing formed with it
// (an address, say) is carried through a loop.
#ifndef KV_OPAQUE_S
#define KV_OPAQUE_S(x) asm("" : "+s"(x))
#define KV_OPAQUE_V(x) asm("" : "+v"(x))
#define KV_FRESH_V(x) asm volatile("" : "+v"(x))
#endif

typedef _Float16 half2v __attribute__((ext_vector_type(2)));

// What the kernels need of gptq_kv_cache and gptq_kv_batch. `shift` is log2
// of the page size, `words` the 32-bit words of one head's codes.
struct KvCache {
  uint32_t* k_codes;
  uint32_t* v_codes;
  uint32_t* k_grid;
  uint32_t* v_grid;
  int64_t n_pages;
  int heads, dim, words, shift;
};
struct KvBatch {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* starts;
  int64_t ld, max_pages, batch, n_tokens;
};

// Sets `*info` (which the caller cleared). Every writer stores the same value.
__device__ __forceinline__ void kv_flag(int32_t* info) {
  if (info) *info = 1;
}

// Page of position `pos` of sequence `b`, or -1 (flagged) where the table
// does not reach or names no page of the cache.
__device__ __forceinline__ int64_t kv_page(const KvCache& c, const KvBatch& q, int64_t b, int64_t pos, int32_t* info) {
  const int64_t at = pos >> c.shift;
  const int64_t id = at < q.max_pages ? int64_t(q.table[b * q.ld + at]) : -1;
  if (id >= 0 && id < c.n_pages) return id;
  kv_flag(info);
  return -1;
}

enum KvState { KV_BEHIND = 0, KV_ABSENT = 1, KV_HELD = 2 };

// Where token t lies. KV_BEHIND: t belongs to no sequence (rows past the last
// one stay as they are). KV_ABSENT: its position is before the sequence's
// start (an idle place of the batch) or on no page. Otherwise `row` is the
// cache row of head 0; head h lies h << shift rows further. Uniform over the
// wave, all of whose lanes take part.
struct KvPlace {
  int state;
  int64_t row;
};
__device__ __forceinline__ KvPlace kv_locate(const KvCache& c, const KvBatch& q, int64_t t, int lane, int32_t* info) {
  KvPlace p{KV_BEHIND, 0};
  int64_t b = t, back = 1;  // sequence, and distance of the token from the sequence's end
  if (q.starts) {
    // The number of starts at or below t, 64 of them at a time. Whatever the
    // array holds, the count stays within its length.
    int64_t n = 0;
    for (int64_t i0 = 0; i0 <= q.batch; i0 += 64) {
      const int64_t i = i0 + lane;
      const uint64_t le = __ballot(i <= q.batch && int64_t(q.starts[i <= q.batch ? i : 0]) <= t);
      n += __popcll(le);
      if (le != ~uint64_t(0)) break;
    }
    b = n - 1;
    if (b < 0 || b >= q.batch) return p;
    back = int64_t(q.starts[b + 1]) - t;
  }
  p.state = KV_ABSENT;
  const int64_t pos = int64_t(q.lens[b]) - back;
  if (pos < 0) return p;
  const int64_t id = kv_page(c, q, b, pos, info);
  if (id < 0) return p;
  p.state = KV_HELD;
  p.row = ((id * c.heads) << c.shift) + (pos & ((int64_t(1) << c.shift) - 1));
  return p;
}

// Grid word: the scale's upper 24 bits (sign, exponent, 15 mantissa bits)
// and the zero point. Sixteen significant bits of the scale keep a quotient
// of a 16-bit input from rounding across a tie (see kv_write); the zero of
// at most 8 bits takes the place of the mantissa's rest, so a head costs one
// word and the scale keeps fp32's whole range.
constexpr uint32_t KV_NAN_GRID = 0x7FC00000u;
__device__ __forceinline__ float kv_scale(uint32_t w) { return __uint_as_float(w & 0xFFFFFF00u); }
template <int BITS>
__device__ __forceinline__ uint32_t kv_zero(uint32_t w) {
  return w & ((1u << BITS) - 1u);
}

struct bf16 {
  uint16_t x;
};
__device__ __forceinline__ float to_f32(_Float16 v) { return float(v); }
__device__ __forceinline__ float to_f32(bf16 v) { return __uint_as_float(uint32_t(v.x) << 16); }
__device__ __forceinline__ float to_f32(float v) { return v; }
// Round to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ _Float16 from_f32<_Float16>(float v) {
  return _Float16(v);
}
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float v) {
  const __bf16 r = __bf16(v);
  bf16 o;
  __builtin_memcpy(&o, &r, 2);
  return o;
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}

// Eight consecutive elements, by 16-byte accesses where `vec` (p 16-byte aligned).
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool vec, float (&x)[8]) {
  T e[8];
  if (vec) {
    uint4 w[sizeof(T) / 2];
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    __builtin_memcpy(e, w, sizeof(e));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = to_f32(e[i]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, bool vec, const float (&x)[8]) {
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(x[i]);
  if (vec) {
    uint4 w[sizeof(T) / 2];
    __builtin_memcpy(w, e, sizeof(e));
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = e[i];
  }
}

// Host side: the checks of the two structs that every entry point makes.
constexpr int64_t KV_MAX_TOKENS = int64_t(1) << 25;  // a launch holds fewer than 2^32 threads, 64 a token

inline int kv_views(const gptq_kv_cache* c, const gptq_kv_batch* b, KvCache* cv, KvBatch* bv) {
  if (!c || !b) return GPTQ_E_INVALID_ARG;
  const void* bufs[4] = {c->k_codes, c->v_codes, c->k_grid, c->v_grid};
  for (const void* p : bufs)
    if (!p || reinterpret_cast<uintptr_t>(p) % 16 != 0) return GPTQ_E_INVALID_ARG;
  if (c->bits != 4 && c->bits != 8) return GPTQ_E_INVALID_ARG;
  if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0) return GPTQ_E_INVALID_ARG;
  if (c->kv_heads < 1 || c->kv_heads > 65535) return GPTQ_E_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0) return GPTQ_E_INVALID_ARG;
  if (c->n_pages < 1 || c->n_pages > INT32_MAX / c->kv_heads) return GPTQ_E_INVALID_ARG;
  if (b->batch < 0 || b->n_tokens < 0 || b->max_pages < 1 || b->ld_table < b->max_pages) return GPTQ_E_INVALID_ARG;
  if (b->batch > KV_MAX_TOKENS || b->n_tokens > KV_MAX_TOKENS || b->max_pages > INT32_MAX) return GPTQ_E_INVALID_ARG;
  if (b->batch > 0 && (!b->table || !b->lens)) return GPTQ_E_INVALID_ARG;
  if (!b->starts && b->n_tokens != b->batch) return GPTQ_E_INVALID_ARG;
  cv->k_codes = c->k_codes;
  cv->v_codes = c->v_codes;
  cv->k_grid = c->k_grid;
  cv->v_grid = c->v_grid;
  cv->n_pages = c->n_pages;
  cv->heads = int(c->kv_heads);
  cv->dim = int(c->head_dim);
  cv->words = int(c->head_dim * c->bits / 32);
  cv->shift = __builtin_ctzll(uint64_t(c->page_size));
  bv->table = b->table;
  bv->lens = b->lens;
  bv->starts = b->starts;
  bv->ld = b->ld_table;
  bv->max_pages = b->max_pages;
  bv->batch = b->batch;
  bv->n_tokens = b->n_tokens;
  return GPTQ_OK;
}

inline size_t kv_elem_bytes(int dtype) { return dtype == GPTQ_F16 || dtype == GPTQ_BF16 ? 2 : dtype == GPTQ_F32 ? 4 : 0; }
// Rows `ld` elements apart that start at p take 16-byte accesses.
inline bool kv_vec16(const void* p, int64_t ld, int dtype) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * int64_t(kv_elem_bytes(dtype))) % 16 == 0;
}

}  // namespace gptq
