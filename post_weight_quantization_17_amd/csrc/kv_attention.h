// Shared parts of the key-value attention kernels (kv_attention.hip has the
// mathematics): the call's arguments, its division into units of work, the
// conversion of codes and the queries.
#pragma once

#include "kv_cache.h"

namespace gptq {

constexpr int ATT_WAVES = 4;
constexpr int ATT_ROWS = 16;                     // query rows of a wave's MFMA
constexpr int ATT_TILE = 32;                     // keys a wave takes at a time
constexpr int ATT_MIN_CHUNK = 256;               // fewest keys of a workgroup when a row's keys are split
constexpr int ATT_UNSPLIT = 512;                 // see cut_call
constexpr int ATT_MAX_TARGET = 4 * 256;          // most workgroups that the keys are split for (Seq)
constexpr int PROMPT_TARGET = 256;               // and in the prompts' kernel
constexpr float ATT_W_TOP = 8.0f;                // log2 of the largest weight after a rescaling
constexpr float ATT_W_LIMIT = 32768.0f;          // a weight above this asks for the next one
constexpr float ATT_S_LEAST = -96.0f;            // log2 of the least step of v that counts in M (kv_attention.hip)
constexpr float ATT_SUM_LIMIT = 0x1p108f;        // a tile's sum of 2^(x - M) above this asks for a rescaling, too
constexpr float ATT_LOWEST = -3.402823466e38f;   // M before the first key
constexpr float LOG2E = 1.44269504088896340736f;

// Division of 0 .. 2^31 - 1 by a number known on the host: with s = ceil(log2
// d) and mul = floor(2^32 (2^s - d) / d) + 1, n / d = (n + floor(n mul / 2^32))
// / 2^s rounded down.
struct Divider {
  uint32_t d, mul, shift;
  static Divider by(uint32_t d) {
    Divider r{d, 0, 0};
    while ((uint64_t(1) << r.shift) < d) ++r.shift;
    r.mul = uint32_t((((uint64_t(1) << r.shift) - d) << 32) / d) + 1;
    return r;
  }
  __device__ __forceinline__ int operator()(int n) const {
    const uint32_t t = uint32_t((uint64_t(uint32_t(n)) * mul) >> 32);
    return int((t + uint32_t(n)) >> shift);
  }
};

struct AttArgs {
  KvCache c;
  KvBatch b;
  const void* q;
  void* out;
  const float* slopes;
  float* part_o;    // [parts][kv_heads][rows][dim]: partial sums
  float2* part_ml;  // [parts][kv_heads][rows]: their reference and weight sum
  int32_t* info;
  int64_t ldq, ldo;
  float scale;  // of the scores, in log2 units
  int ratio;    // query heads that share a key-value head
  int q_dtype, out_dtype, q_vec, out_vec;
  int block_shift; // log2 of a row block's query rows
  Divider by_heads, by_ratio;  // kv_heads, ratio
  int per_token;   // row blocks of one token, where each sequence has one
  int rows;     // most of them that a call has: those of a part
  int splits;   // 0: no row block's keys are split
  int units;    // of the launch
  int parts;    // that the workspace holds
  int target;   // workgroups that the keys are split for
};

__device__ __forceinline__ void store_out(const AttArgs& a, int64_t at, float v) {
  if (a.out_dtype == GPTQ_F16)
    static_cast<_Float16*>(a.out)[at] = from_f32<_Float16>(v);
  else if (a.out_dtype == GPTQ_BF16)
    static_cast<bf16*>(a.out)[at] = from_f32<bf16>(v);
  else
    static_cast<float*>(a.out)[at] = v;
}

// The row blocks of 2^shift rows of a sequence with n new tokens.
__host__ __device__ __forceinline__ int64_t row_blocks(int64_t n, int ratio, int shift) {
  return (n * ratio + (int64_t(1) << shift) - 1) >> shift;
}

// A call's work is cut into units: one row block (of one key-value head) over
// one chunk of its sequence's keys. The chunk is the same for all sequences,
// so that units take about the same time however ragged the batch is: the
// keys of all row blocks over the workgroups that the GPU is to be filled
// with, in whole tiles of the 4 waves. Lengths are device data, so every
// workgroup works the chunk out for itself, from the same numbers in the same
// order. A sequence has ceil(len / chunk) units a row block (at least one,
// which writes the zeros of rows without keys); those past a causal row
// block's last key have nothing to do.
//
// The host's bound of the units (call_units) holds because each sequence has
// at most len / chunk + 1 a row block, and chunk is at least the mean share;
// where a row block has several, at most 2 len / chunk: those are the parts.
// The launch has fewer than 2^24 row blocks, so n * ratio fits 32 bits;
// lengths are int32, so positions and their sums here do, too.
struct Seq {
  int b;       // sequence, -1: none
  int t0;      // its first token
  int n;       // its new tokens
  int rb;      // row block within it
  int split;   // chunk of its keys
  int splits;  // chunks that the sequence's keys are cut into
  int first;   // part of the row block's first chunk, where it has several
  int64_t len;
  uint32_t chunk;
};

// Tokens and keys of sequence b (no tokens where starts are out of order).
struct Span {
  int t0, n;
  int64_t len;
};
__device__ __forceinline__ Span seq_span(const KvBatch& q, int64_t b) {
  Span s{int(b), 0, 0};
  if (b >= q.batch) return s;
  s.len = q.lens[b];
  s.n = 1;
  if (q.starts) {
    const int64_t t0 = q.starts[b], n = int64_t(q.starts[b + 1]) - t0;
    const bool ok = n >= 0 && t0 >= 0 && t0 + n <= q.n_tokens;
    s.t0 = ok ? int(t0) : 0;
    s.n = ok ? int(n) : 0;
  }
  return s;
}
__device__ __forceinline__ uint32_t cached(int64_t len, int64_t cap) { return uint32_t(len < 0 ? 0 : len > cap ? cap : len); }

// Inclusive prefix sums over the wave, by DPP adds: shifts by 1, 2, 4 and 8
// within the rows of 16 lanes, then the rows' last sums to the rows behind.
template <typename T, int CTRL, int ROWS>
__device__ __forceinline__ T dpp_or_zero(T v) {
  int w, r;
  __builtin_memcpy(&w, &v, 4);
  r = __builtin_amdgcn_update_dpp(0, w, CTRL, ROWS, 0xf, false);
  __builtin_memcpy(&v, &r, 4);
  return v;
}
template <typename T>
__device__ __forceinline__ T wave_prefix(T v) {
  v += dpp_or_zero<T, 0x111, 0xf>(v);
  v += dpp_or_zero<T, 0x112, 0xf>(v);
  v += dpp_or_zero<T, 0x114, 0xf>(v);
  v += dpp_or_zero<T, 0x118, 0xf>(v);
  v += dpp_or_zero<T, 0x142, 0xa>(v);
  v += dpp_or_zero<T, 0x143, 0xc>(v);
  return v;
}

// The unit number `at` (JOIN = false), or the row block number `at` of those
// with several units (JOIN = true). Uniform over the wave, all of whose lanes
// take part.
template <bool JOIN>
__device__ __forceinline__ Seq find_unit(const AttArgs& a, int at, int lane) {
  const KvBatch& q = a.b;
  const int64_t cap = q.max_pages << a.c.shift;
  Seq r{-1, 0, 0, 0, 0, 1, 0, 0, 0xFFFFFF80u};  // a chunk that holds any length
  if (a.splits) {
    float work = 0.0f;
    for (int64_t b0 = 0; b0 < q.batch; b0 += 64) {
      const Span s = seq_span(q, b0 + lane);
      work += float(row_blocks(s.n, a.ratio, a.block_shift)) * float(cached(s.len, cap));
    }
    work = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wave_prefix(work)), 63));
    constexpr uint32_t step = ATT_WAVES * ATT_TILE;
    const float share = fminf(work * float(a.c.heads) / float(a.target), 2.0e9f);
    const uint32_t chunk = (uint32_t(share) + step) / step * step;
    r.chunk = chunk < ATT_MIN_CHUNK ? ATT_MIN_CHUNK : chunk;
  }
  int before = 0, parts_before = 0;  // of the sequences passed
  for (int64_t b0 = 0; b0 < q.batch; b0 += 64) {
    const Span s = seq_span(q, b0 + lane);
    const uint32_t keys = cached(s.len, cap);
    const int splits = a.splits && keys > r.chunk ? int((keys - 1) / r.chunk) + 1 : 1;
    const int blocks = int(row_blocks(s.n, a.ratio, a.block_shift));
    // A sum past 2^24 is past the launch, whatever the arrays hold.
    const int64_t all = int64_t(blocks) * splits;
    const int units = int(all < (1 << 24) ? all : (1 << 24));
    const int mine = !JOIN ? units : splits > 1 ? blocks : 0;
    const int parts = splits > 1 ? units : 0;
    const int sum = wave_prefix(mine), parts_sum = wave_prefix(parts);
    const uint64_t past = __ballot(sum > at - before);
    if (past != 0) {
      const int src = __ffsll((unsigned long long)past) - 1;
      const auto take = [&](int v) { return __builtin_amdgcn_readlane(v, src); };
      r.b = int(b0) + src;
      r.t0 = take(s.t0);
      r.n = take(s.n);
      r.len = take(int(s.len));
      r.splits = take(splits);
      const int n_blocks = take(blocks), k = at - before - take(sum - mine);
      // The last row blocks see the most keys and come first.
      const int back = JOIN ? k : k / r.splits;
      r.rb = n_blocks - 1 - back;
      r.split = JOIN ? 0 : k - back * r.splits;
      r.first = parts_before + take(parts_sum - parts) + back * r.splits;
      return r;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
    parts_before += __builtin_amdgcn_readlane(parts_sum, 63);
    if (before > at || parts_before > (1 << 24)) break;
  }
  return r;
}

// Keys that new token i of n of a sequence of `len` tokens sees, `cap` of
// which the table reaches.
__device__ __forceinline__ uint32_t keys_seen(int64_t len, int n, int i, int64_t cap) {
  const int64_t end = len - n + i + 1;
  return uint32_t(end < 0 ? 0 : end > cap ? cap : end);
}
__device__ __forceinline__ int block_last_row(const AttArgs& a, int n, int rb) {
  const int last = ((rb + 1) << a.block_shift) - 1, rows = n * a.ratio;
  return last < rows ? last : rows - 1;
}

__device__ __forceinline__ uint32_t as_u32(half2v v) {
  uint32_t r;
  __builtin_memcpy(&r, &v, 4);
  return r;
}
__device__ __forceinline__ half2v as_half2(uint32_t v) {
  half2v r;
  __builtin_memcpy(&r, &v, 4);
  return r;
}
__device__ __forceinline__ half8 as_half8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t w[4] = {a, b, c, d};
  half8 r;
  __builtin_memcpy(&r, w, 16);
  return r;
}

// What a code is offset by in its fp16 half, the bits of that half, and the
// position of the code in it.
template <int BITS>
struct Half {
  static constexpr float off = BITS == 4 ? 64.0f : 1024.0f;
  static constexpr uint32_t magic = BITS == 4 ? 0x54005400u : 0x64006400u;
  static constexpr int at = BITS == 4 ? 4 : 0;
};

// The conversion's constants, kept in registers: a mask in an SGPR and the
// exponent pattern in a VGPR make mask-and-merge one v_and_or_b32, which
// takes no literals.
struct Consts {
  uint32_t mask, magic;
};
template <int BITS>
__device__ __forceinline__ Consts conversion_consts() {
  Consts k{0x00F000F0u, Half<BITS>::magic};
  KV_OPAQUE_S(k.mask);
  KV_OPAQUE_V(k.magic);
  return k;
}

// 4-bit codes: code i (0..3) of each 16-bit half of w, as two halves 64 + c.
template <int I>
__device__ __forceinline__ uint32_t nibbles(uint32_t w, const Consts& k) {
  constexpr int up = 4 - 4 * I;
  return ((up > 0 ? w << up : w >> -up) & k.mask) | k.magic;
}
// 8-bit codes: bytes A and B of w, as two halves 1024 + c.
template <int A, int B>
__device__ __forceinline__ uint32_t byte_pair(uint32_t w, const Consts& k) {
  return __builtin_amdgcn_perm(k.magic, w, 0x05000500u | A | B << 16);
}

// The 8 codes of a lane's k-slots in one MFMA of the first product. 4 bits:
// one word, in the order 0 4 1 5 2 6 3 7; 8 bits: two words, in order.
template <int BITS>
struct KeyOrder {
  static constexpr int code(int i) { return BITS == 4 ? (i % 2) * 4 + i / 2 : i; }
};
template <int BITS>
__device__ __forceinline__ void key_codes(const uint32_t* w, uint32_t (&h)[4], const Consts& k) {
  if constexpr (BITS == 4) {
    h[0] = nibbles<0>(w[0], k);
    h[1] = nibbles<1>(w[0], k);
    h[2] = nibbles<2>(w[0], k);
    h[3] = nibbles<3>(w[0], k);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      h[2 * i] = byte_pair<0, 1>(w[i], k);
      h[2 * i + 1] = byte_pair<2, 3>(w[i], k);
    }
  }
}

// N words at p, which is aligned to the largest power of two that divides
// their size, 16 bytes at most.
template <int N>
__device__ __forceinline__ void load_words(const char* p, uint32_t* w) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint2 v = reinterpret_cast<const uint2*>(p)[i];
      w[2 * i] = v.x, w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}

// Where 16 keys of a head lie, as byte offsets into the codes and the grids
// (the same for k and v). The host has checked that pages times heads fit 31
// bits, so one 32-bit product and one widening product each suffice. Keys
// outside the cache's pages (flagged where they count, p < k1) get the first
// page's: those are there to be read, and are masked.
struct Place16 {
  uint64_t codes, grid;
  uint32_t ok;
  __device__ __forceinline__ Place16 next(int words) const { return Place16{codes + 64u * uint32_t(words), grid + 64u, ok}; }
};
__device__ __forceinline__ Place16 place16(const KvCache& c, int32_t* info, int kv, int page, uint32_t p, uint32_t k1) {
  uint32_t id = uint32_t(__builtin_amdgcn_readfirstlane(page));
  const uint32_t ok = id < uint32_t(c.n_pages);
  if (!ok) {
    if (p < k1) kv_flag(info);
    id = 0;
  }
  const uint32_t head = id * uint32_t(c.heads) + uint32_t(kv), in = p & ((1u << c.shift) - 1);
  const uint32_t row = 4u * uint32_t(c.words);
  return Place16{uint64_t(head) * (row << c.shift) + in * row, uint64_t(head) * (4u << c.shift) + 4u * in, ok};
}

// A lane's part of a query row as the B operand of the first product: its
// blocks of 8 elements, in the order of the codes, scaled to a largest element
// of 2^13 to 2^14 and split in two parts where SPLIT; their sum, for the
// codes' offset; and what turns the product into a score in log2 units.
template <int DP, bool FULL>
__device__ __forceinline__ int lane_block(int g, int j) {
  return FULL ? g * (DP / 32) + j : 4 * j + g;
}
template <int BITS, int DP, bool FULL, bool SPLIT>
struct Query {
  static constexpr int NJ = DP / 32;
  half8 h[NJ], l[NJ];
  float sum, scale;

  __device__ __forceinline__ void load(const AttArgs& a, bool live, int64_t token, int head, int g) {
    float f[NJ][8];
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[j][e] = 0.0f;
      const int d0 = 8 * lane_block<DP, FULL>(g, j);
      if (live && d0 < a.c.dim) {
        const int64_t at = token * a.ldq + int64_t(head) * a.c.dim + d0;
        if (a.q_dtype == GPTQ_F16)
          load8(static_cast<const _Float16*>(a.q) + at, a.q_vec, f[j]);
        else if (a.q_dtype == GPTQ_BF16)
          load8(static_cast<const bf16*>(a.q) + at, a.q_vec, f[j]);
        else
          load8(static_cast<const float*>(a.q) + at, a.q_vec, f[j]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[j][e]));
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    int ex = int(__float_as_uint(top) >> 23) - 127;
    if (ex > 127 || top == 0.0f) ex = 13;  // nothing to scale, or an infinity
    scale = ldexpf(a.scale, ex - 13);
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = ldexpf(f[j][KeyOrder<BITS>::code(e)], 13 - ex);
        h[j][e] = _Float16(s);
        sum += float(h[j][e]);
        if constexpr (SPLIT) l[j][e] = _Float16(s - float(h[j][e]));
      }
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
  }
};

// The prompts' kernel (kv_prompt.hip).
constexpr int PROMPT_BLOCK = 128;  // query rows of its row blocks
int launch_prompt(const AttArgs& a, int bits, bool split, hipStream_t s);

}  // namespace gptq
