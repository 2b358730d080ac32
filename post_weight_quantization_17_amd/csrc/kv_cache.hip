// Quantised key-value cache: storing tokens and reading them back.
//
// The grid is the framework's min-max grid (astro-blog survey, section 1.2;
// aiqz.cc, section 分组方案) with one group per token and head:
//   lo = min(0, min x), hi = max(0, max x), s = (hi - lo) / (2^b - 1),
//   z = rint(-lo / s), c = clamp(rint(x / s) + z, 0, 2^b - 1), x^ = s (c - z).
//
// Rounding. hi - lo and the division by 2^b - 1 are fp32 operations; s is
// then rounded to 16 significant bits (ties to even), which is what the grid
// word holds, so codes and reader use the same s. rint is taken of the real
// quotient Q = x / s. It is formed as q = x r, q' = q + (x - q s) r with r =
// rcp(s) and FMAs: the residual x - q s is exact, so q' is the rounding of Q
// (1 + d), |d| < 2^-45. For a 16-bit x (at most 11 significant bits) that
// decides as Q does: Q differs from a half-integer k + 1/2 < 256 by |2x - s
// (2k+1)| / (2s), which is 0 (then q' is the half-integer) or at least ulp(s)
// / (2s) > 2^-17 (an x of s/4 or more has no bit below ulp(s)), more than half
// an fp32 step below 256. An fp32 x can lie closer: where q' comes out a
// half-integer the sign of its residual decides. s = range / (2^b - 1) is
// formed alike with the constant's reciprocal; no quotient by 15 or 255 lies
// within 2^-29 of a rounding boundary, so it is the correctly rounded one.
// Residuals are exact while s is above 2^-90; smaller ones are scaled up.
//
// Measured (large copy 5.1 TB/s): 65536 tokens of 32 heads of 128, 8 bits, read
// back to bf16 in 311 us (5.2 TB/s); 39680 tokens of 32 heads of 80, 4 bits, from
// bf16 stored in 138 to 158 us (3.3 to 3.8 TB/s, the 16-lane rows of the range
// hold 10 busy lanes) and read back in 135 us; 2048 tokens of 96 heads, 8 bits,
// stored in 38 us (4.0 TB/s). A token: 3 us, the launch and three dependent
// loads (length, page, place).
//
// q' + 1.5 * 2^23 is rint(q') in its low bits; those are clamped as floats and
// gathered by shift-and-add, the zero point and the constant's own bits once
// for all of a word's codes.
#include "kv_cache.h"

namespace gptq {
namespace {

constexpr int KV_WAVES = 4;  // waves per workgroup, one token each
constexpr int64_t KV_RESIDENT_WAVES = 256 * 32;

// Eight elements as loaded, and the range of a head vector over its LPR
// lanes. Lanes past the head's end hold zeros, which leave the range as it
// is. Maxima are taken on the bit patterns: as signed integers the largest is
// the largest number (or negative), as unsigned ones the most negative number
// (or positive); infinities and NaNs lie past every finite number in both.
struct Range {
  float lo, hi;
  bool finite;
};
template <int LPR, typename F>
__device__ __forceinline__ int row_reduce(int v, F op) {
  if constexpr (LPR >= 2) v = op(v, __builtin_amdgcn_mov_dpp(v, 0xB1, 0xf, 0xf, false));   // quad_perm [1,0,3,2]
  if constexpr (LPR >= 4) v = op(v, __builtin_amdgcn_mov_dpp(v, 0x4E, 0xf, 0xf, false));   // quad_perm [2,3,0,1]
  if constexpr (LPR >= 8) v = op(v, __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, false));  // row_half_mirror
  if constexpr (LPR >= 16) v = op(v, __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, false)); // row_mirror
  if constexpr (LPR >= 32) v = op(v, __shfl_xor(v, 16));
  return v;
}

typedef short short2v __attribute__((ext_vector_type(2)));
typedef unsigned short ushort2v __attribute__((ext_vector_type(2)));
template <typename T>
__device__ __forceinline__ T as_type(uint32_t w) {
  T r;
  __builtin_memcpy(&r, &w, 4);
  return r;
}
template <typename T>
__device__ __forceinline__ uint32_t bits_of(T v) {
  uint32_t w;
  __builtin_memcpy(&w, &v, 4);
  return w;
}
__device__ __forceinline__ uint32_t max2_i16(uint32_t a, uint32_t b) {
  return bits_of(__builtin_elementwise_max(as_type<short2v>(a), as_type<short2v>(b)));
}
__device__ __forceinline__ uint32_t max2_u16(uint32_t a, uint32_t b) {
  return bits_of(__builtin_elementwise_max(as_type<ushort2v>(a), as_type<ushort2v>(b)));
}

template <typename T>
struct Raw8 {  // 16-bit types
  uint32_t w[4];
  __device__ __forceinline__ void get(float (&x)[8]) const {
    T e[8];
    __builtin_memcpy(e, w, 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(e[i]);
  }
  template <int LPR>
  __device__ __forceinline__ Range range() const {
    const uint32_t up = max2_i16(max2_i16(w[0], w[1]), max2_i16(w[2], w[3]));
    const uint32_t down = max2_u16(max2_u16(w[0], w[1]), max2_u16(w[2], w[3])) ^ 0x80008000u;  // now in signed order
    // The larger of each one's halves, side by side: largest | most negative.
    const uint32_t two = max2_i16((up & 0xFFFFu) | down << 16, (up >> 16) | (down & 0xFFFF0000u));
    const uint32_t m = uint32_t(row_reduce<LPR>(int(two), [](int a, int b) { return int(max2_i16(uint32_t(a), uint32_t(b))); }));
    const uint32_t h = m & 0xFFFFu, l = (m >> 16) ^ 0x8000u;
    constexpr uint32_t inf = __is_same(T, _Float16) ? 0x7C00u : 0x7F80u;
    const uint16_t hb = uint16_t(h & 0x8000u ? 0u : h), lb = uint16_t(l & 0x8000u ? l : 0u);
    T ht, lt;
    __builtin_memcpy(&ht, &hb, 2);
    __builtin_memcpy(&lt, &lb, 2);
    return Range{to_f32(lt), to_f32(ht), hb < inf && lb < (0x8000u | inf)};
  }
};
template <>
struct Raw8<float> {
  uint32_t w[8];
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
  template <int LPR>
  __device__ __forceinline__ Range range() const {
    int up = 0;
    uint32_t down = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      up = int(w[i]) > up ? int(w[i]) : up;
      down = w[i] > down ? w[i] : down;
    }
    up = row_reduce<LPR>(up, [](int a, int b) { return a > b ? a : b; });
    down = uint32_t(row_reduce<LPR>(int(down), [](int a, int b) { return int(uint32_t(a) > uint32_t(b) ? uint32_t(a) : uint32_t(b)); }));
    const float lo = __uint_as_float(down & 0x80000000u ? down : 0u);
    return Range{lo, __int_as_float(up), uint32_t(up) < 0x7F800000u && down < 0xFF800000u};
  }
};

template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* p, bool vec) {
  Raw8<T> r;
  constexpr int N = sizeof(r.w) / 16;
  if (vec) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
  } else {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = p[i];
    __builtin_memcpy(r.w, e, sizeof(r.w));
  }
  return r;
}

constexpr float KV_ROUND = 12582912.0f;  // 1.5 * 2^23

// KV_ROUND + rint(x / s), r = rcp(s).
template <bool EXACT>
__device__ __forceinline__ float rounded_quotient(float x, float s, float r) {
  float q = x * r;
  q = fmaf(fmaf(-q, s, x), r, q);
  float y = q + KV_ROUND;
  if constexpr (EXACT) {
    if (fabsf(q - (y - KV_ROUND)) == 0.5f) {
      const float res = fmaf(-q, s, x);
      if (res != 0.0f) y = KV_ROUND + (res < 0.0f ? floorf(q) : ceilf(q));
    }
  }
  return y;
}

// One head vector, 8 elements a lane on LPR lanes: grid word and codes.
template <typename T, int LPR, int BITS>
__device__ __forceinline__ uint32_t quantise8(const Raw8<T>& raw, uint32_t (&words)[BITS / 4]) {
  constexpr float top = float((1 << BITS) - 1);
  constexpr bool tiny = !__is_same(T, _Float16);  // fp16's s is above 2^-33
  constexpr bool exact = __is_same(T, float);
  const Range g = raw.template range<LPR>();
  float x[8];
  raw.get(x);
  float lo = g.lo;
  const float range = g.hi - g.lo;
  const bool bad = !g.finite || !(range <= 3.402823466e38f);
  float s = range * (1.0f / top);
  s = fmaf(fmaf(-s, top, range), 1.0f / top, s);
  bool small = false;
  if constexpr (tiny) {
    small = range < 0x1p-80f;
    if (__any(small)) s = small ? range / top : s;
  }
  if (s < 0x1p-126f) {  // an all-zero vector, or one below every normal step: the grid of [-1, 1]
    s = 2.0f / top;
    lo = -1.0f;
    small = false;
  }
  uint32_t sb = __float_as_uint(s);
  sb = (sb + 0x7Fu + ((sb >> 8) & 1u)) & 0xFFFFFF00u;
  s = __uint_as_float(sb);
  if constexpr (tiny) {
    if (__any(small)) {
      const float p = small ? 0x1p100f : 1.0f;
      s *= p;
      lo *= p;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= p;
    }
  }
  const float r = __builtin_amdgcn_rcpf(s);
  const float z = rounded_quotient<exact>(-lo, s, r) - KV_ROUND;
  const float least = KV_ROUND - z, most = least + top;
  const uint32_t zi = uint32_t(int(bad ? 0.0f : z));
  constexpr int per = 32 / BITS;
#pragma unroll
  for (int h = 0; h < BITS / 4; ++h) {
    uint32_t w = 0, each = 0, base = 0;
#pragma unroll
    for (int i = per - 1; i >= 0; --i) {
      const float y = __builtin_amdgcn_fmed3f(rounded_quotient<exact>(x[per * h + i], s, r), least, most);
      w = (w << BITS) + __float_as_uint(y);
      each = each << BITS | 1u;
      base = (base << BITS) + 0x4B400000u;  // the bits of KV_ROUND
    }
    words[h] = bad ? 0u : w - base + zi * each;
  }
  return bad ? KV_NAN_GRID : sb | zi;
}

// Wave = one token and IT groups of 64 / LPR of its heads (K and V), a lane
// 8 elements of each: 16-byte loads, one or two words of codes. All loads
// are issued before the token's place is looked up.
template <typename T, int LPR, int BITS, int IT>
__global__ void __launch_bounds__(64 * KV_WAVES)
kv_write(KvCache c, KvBatch q, const T* __restrict__ k, const T* __restrict__ v, int64_t ldk, int64_t ldv, int vec,
         int32_t* __restrict__ info) {
  constexpr int W = BITS / 4, HEADS = 64 / LPR;
  const int lane = threadIdx.x % 64;
  const int64_t t = int64_t(blockIdx.x) * KV_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  if (t >= q.n_tokens) return;  // whole waves; no barrier follows
  const int e = lane % LPR;
  const int h0 = int(blockIdx.y) * HEADS * IT + lane / LPR;
  Raw8<T> x[IT][2] = {};
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int h = h0 + HEADS * i;
    if (h < c.heads && 8 * e < c.dim) {
      x[i][0] = load_raw8(k + t * ldk + (h * c.dim + 8 * e), vec);
      x[i][1] = load_raw8(v + t * ldv + (h * c.dim + 8 * e), vec);
    }
  }
  const KvPlace p = kv_locate(c, q, t, lane, info);
  if (p.state != KV_HELD) return;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int h = h0 + HEADS * i;
    const int64_t row = p.row + (int64_t(h) << c.shift);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint32_t w[W];
      const uint32_t grid = quantise8<T, LPR, BITS>(x[i][kv], w);
      if (h < c.heads && 8 * e < c.dim) {
        uint32_t* codes = (kv ? c.v_codes : c.k_codes) + row * c.words + W * e;
        if constexpr (W == 1)
          *codes = w[0];
        else
          *reinterpret_cast<uint2*>(codes) = uint2{w[0], w[1]};
        if (e == 0) (kv ? c.v_grid : c.k_grid)[row] = grid;
      }
    }
  }
}

template <int BITS>
__device__ __forceinline__ void values8(const uint32_t (&w)[BITS / 4], uint32_t grid, float (&x)[8]) {
  const float s = kv_scale(grid), z = float(kv_zero<BITS>(grid));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t code = BITS == 4 ? (w[0] >> (4 * i)) & 15u : (w[i / 4] >> (8 * (i % 4))) & 255u;
    x[i] = s * (float(code) - z);
  }
}

// Wave = one token and IT times 64 groups of 8 elements of its row (K and
// V), whatever heads they fall into: every lane has work at any head_dim.
template <typename T, int BITS, int IT>
__global__ void __launch_bounds__(64 * KV_WAVES)
kv_read(KvCache c, KvBatch q, T* __restrict__ k, T* __restrict__ v, int64_t ldk, int64_t ldv, int vec,
        int32_t* __restrict__ info) {
  constexpr int W = BITS / 4;
  const int lane = threadIdx.x % 64;
  const int64_t t = int64_t(blockIdx.x) * KV_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  if (t >= q.n_tokens) return;
  const int per = c.dim / 8, groups = c.heads * per;
  const int g0 = int(blockIdx.y) * 64 * IT + lane;
  const KvPlace p = kv_locate(c, q, t, lane, info);
  if (p.state == KV_BEHIND) return;
  uint32_t w[IT][2][W], grid[IT][2];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int g = g0 + 64 * i;
    const int h = int(unsigned(g) / unsigned(per)), e = g - h * per;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      grid[i][kv] = 0;  // a row without a token reads as zeros
#pragma unroll
      for (int j = 0; j < W; ++j) w[i][kv][j] = 0;
      if (p.state == KV_HELD && g < groups) {
        const int64_t row = p.row + (int64_t(h) << c.shift);
        const uint32_t* codes = (kv ? c.v_codes : c.k_codes) + row * c.words + W * e;
        if constexpr (W == 1) {
          w[i][kv][0] = *codes;
        } else {
          const uint2 two = *reinterpret_cast<const uint2*>(codes);
          w[i][kv][0] = two.x, w[i][kv][1] = two.y;
        }
        grid[i][kv] = (kv ? c.v_grid : c.k_grid)[row];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int g = g0 + 64 * i;
    if (g >= groups) continue;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float x[8];
      values8<BITS>(w[i][kv], grid[i][kv], x);
      store8((kv ? v + t * ldv : k + t * ldk) + 8 * g, vec, x);
    }
  }
}

// Calls f with the kernel's lanes per head row: the power of two that holds
// head_dim / 8 of them.
template <typename F>
int with_lanes(int dim, F f) {
  if (dim <= 16) return f(std::integral_constant<int, 2>{});
  if (dim <= 32) return f(std::integral_constant<int, 4>{});
  if (dim <= 64) return f(std::integral_constant<int, 8>{});
  if (dim <= 128) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}
template <typename F>
int with_type(int dtype, F f) {
  if (dtype == GPTQ_F16) return f(_Float16{});
  if (dtype == GPTQ_BF16) return f(bf16{});
  return f(float{});
}
template <typename F>
int with_bits(int bits, F f) {
  return bits == 4 ? f(std::integral_constant<int, 4>{}) : f(std::integral_constant<int, 8>{});
}

// Calls f with the groups of a token that a wave takes, and the grid: one
// while that leaves fewer waves than the GPU holds at once (a small call is
// all latency), else up to four, so that a wave's look-ups and its memory
// latency are paid for more bytes.
template <typename F>
int with_groups(int64_t n_tokens, int groups, F f) {
  const unsigned x = unsigned((n_tokens + KV_WAVES - 1) / KV_WAVES);
  const auto grid = [&](int it) { return dim3(x, unsigned((groups + it - 1) / it)); };
  if (n_tokens * groups <= KV_RESIDENT_WAVES || groups == 1) return f(std::integral_constant<int, 1>{}, grid(1));
  if (groups <= 2) return f(std::integral_constant<int, 2>{}, grid(2));
  return f(std::integral_constant<int, 4>{}, grid(4));
}

// What both entry points check of the dense side: `held` values a token,
// rows ldk and ldv apart.
int check_dense(const KvCache& c, const KvBatch& b, const void* k, const void* v, int dtype, int64_t ldk, int64_t ldv) {
  const size_t eb = kv_elem_bytes(dtype);
  const int64_t row = int64_t(c.heads) * c.dim;
  if (eb == 0 || ldk < row || ldv < row || ldk > (int64_t(1) << 40) || ldv > (int64_t(1) << 40))
    return GPTQ_E_INVALID_ARG;
  if (b.n_tokens > 0 && (!k || !v)) return GPTQ_E_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(k) % eb != 0 || reinterpret_cast<uintptr_t>(v) % eb != 0) return GPTQ_E_INVALID_ARG;
  return GPTQ_OK;
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" int gptq_kv_cache_write(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const void* k,
                                   const void* v, int dtype, int64_t ldk, int64_t ldv, int32_t* info, void* stream) {
  KvCache c;
  KvBatch b;
  int st = kv_views(cache, batch, &c, &b);
  if (st == GPTQ_OK) st = check_dense(c, b, k, v, dtype, ldk, ldv);
  if (st != GPTQ_OK || b.n_tokens == 0 || b.batch == 0) return st;
  const int vec = kv_vec16(k, ldk, dtype) && kv_vec16(v, ldv, dtype);
  hipStream_t s = as_stream(stream);
  return with_type(dtype, [&](auto ty) {
    return with_lanes(c.dim, [&](auto lpr) {
      return with_bits(cache->bits, [&](auto bits) {
        return with_groups(b.n_tokens, (c.heads + 64 / lpr.value - 1) / (64 / lpr.value), [&](auto it, dim3 grid) {
          using T = decltype(ty);
          hipLaunchKernelGGL((kv_write<T, lpr.value, bits.value, it.value>), grid, dim3(64 * KV_WAVES), 0, s, c, b,
                             static_cast<const T*>(k), static_cast<const T*>(v), ldk, ldv, vec, info);
          return launch_status();
        });
      });
    });
  });
}

extern "C" int gptq_kv_cache_read(const gptq_kv_cache* cache, const gptq_kv_batch* batch, void* k, void* v, int dtype,
                                  int64_t ldk, int64_t ldv, int32_t* info, void* stream) {
  KvCache c;
  KvBatch b;
  int st = kv_views(cache, batch, &c, &b);
  if (st == GPTQ_OK) st = check_dense(c, b, k, v, dtype, ldk, ldv);
  if (st != GPTQ_OK || b.n_tokens == 0 || b.batch == 0) return st;
  const int vec = kv_vec16(k, ldk, dtype) && kv_vec16(v, ldv, dtype);
  hipStream_t s = as_stream(stream);
  return with_type(dtype, [&](auto ty) {
    return with_bits(cache->bits, [&](auto bits) {
      return with_groups(b.n_tokens, (c.heads * (c.dim / 8) + 63) / 64, [&](auto it, dim3 grid) {
        using T = decltype(ty);
        hipLaunchKernelGGL((kv_read<T, bits.value, it.value>), grid, dim3(64 * KV_WAVES), 0, s, c, b,
                           static_cast<T*>(k), static_cast<T*>(v), ldk, ldv, vec, info);
        return launch_status();
      });
    });
  });
}
