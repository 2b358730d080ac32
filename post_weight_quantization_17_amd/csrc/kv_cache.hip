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
// quotient x / s. For a 16-bit x (at most 11 significant bits) the correctly
// rounded fp32 quotient decides alike: x / s differs from a half-integer
// k + 1/2 < 256 by |2x - s (2k+1)| / (2s), which is 0 or at least
// ulp(s) / (2s) > 2^-17 (x of at least s/4 has no bit below ulp(s)), more than
// half an fp32 step below 256; and a tie comes out exactly. An fp32 x can lie
// closer, so a quotient that comes out a half-integer is put right by the
// sign of its residual. The quotient is x * (1/s) with one residual step: 1/s
// correctly rounded and two FMAs give the correctly rounded quotient; x and s
// are scaled by s's power of two first where the type's range asks for it.
#include "kv_cache.h"

namespace gptq {
namespace {

constexpr int KV_WAVES = 4;  // waves per workgroup, one token each

template <int LPR>
__device__ __forceinline__ float row_min(float v) {
  if constexpr (LPR >= 2) v = fminf(v, dpp_xor1(v));
  if constexpr (LPR >= 4) v = fminf(v, dpp_xor2(v));
  if constexpr (LPR >= 8) v = fminf(v, dpp_half_mirror(v));
  if constexpr (LPR >= 16) v = fminf(v, dpp_mirror(v));
  if constexpr (LPR >= 32) v = fminf(v, __shfl_xor(v, 16));
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (LPR >= 2) v = fmaxf(v, dpp_xor1(v));
  if constexpr (LPR >= 4) v = fmaxf(v, dpp_xor2(v));
  if constexpr (LPR >= 8) v = fmaxf(v, dpp_half_mirror(v));
  if constexpr (LPR >= 16) v = fmaxf(v, dpp_mirror(v));
  if constexpr (LPR >= 32) v = fmaxf(v, __shfl_xor(v, 16));
  return v;
}

// rint(x / s) as above, for s = m (already scaled into [1, 2) where the type
// needs it, and x with it) and r = 1 / m correctly rounded.
template <bool EXACT>
__device__ __forceinline__ float rint_quotient(float x, float m, float r) {
  float q = x * r;
  q = fmaf(fmaf(-q, m, x), r, q);
  float k = rintf(q);
  if constexpr (EXACT) {
    const float res = fmaf(-q, m, x);
    if (fabsf(q - k) == 0.5f && res != 0.0f) k = res < 0.0f ? floorf(q) : ceilf(q);
  }
  return k;
}

// One head vector, 8 elements a lane on LPR lanes (lanes past the head's end
// hold zeros, which leave the range as it is): grid word and codes.
template <typename T, int LPR, int BITS>
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], uint32_t (&words)[BITS / 4], int lane) {
  constexpr float top = float((1 << BITS) - 1);
  constexpr bool wide = !__is_same(T, _Float16);  // exponents that 1 / s or a residual could leave
  constexpr bool exact = __is_same(T, float);
  float lo = 0.0f, hi = 0.0f, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    sum += x[i];
  }
  // A NaN shows in the sum; an infinity in the range.
  const uint64_t nan_lanes = __ballot(sum != sum);
  lo = row_min<LPR>(lo);
  hi = row_max<LPR>(hi);
  const uint64_t row_lanes = (LPR == 64 ? ~uint64_t(0) : (uint64_t(1) << LPR) - 1) << (lane & ~(LPR - 1));
  const float range = hi - lo;
  const bool bad = (nan_lanes & row_lanes) != 0 || !(range <= 3.402823466e38f);
  float s = range / top;
  if (s < 1.17549435e-38f) {  // an all-zero vector, or one below every normal step: the grid of [-1, 1]
    s = 2.0f / top;
    lo = -1.0f;
  }
  uint32_t sb = __float_as_uint(s);
  sb = (sb + 0x7Fu + ((sb >> 8) & 1u)) & 0xFFFFFF00u;
  s = __uint_as_float(sb);
  float m = s, p2 = 1.0f;
  if constexpr (wide) {
    m = __uint_as_float((sb & 0x007FFFFFu) | 0x3F800000u);
    p2 = __uint_as_float(0x7F000000u - (sb & 0x7F800000u));  // 2^-exponent: s is normal and below 2^127
  }
  const float r = 1.0f / m;
  const float z = rint_quotient<exact>(-lo * p2, m, r);
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i] = fminf(fmaxf(rint_quotient<exact>(wide ? x[i] * p2 : x[i], m, r) + z, 0.0f), top);
  if constexpr (BITS == 4) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= uint32_t(fmaf(c[2 * i + 1], 16.0f, c[2 * i])) << (8 * i);
    words[0] = bad ? 0u : w;
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) w |= uint32_t(c[4 * h + i]) << (8 * i);
      words[h] = bad ? 0u : w;
    }
  }
  return bad ? KV_NAN_GRID : sb | uint32_t(z);
}

// Wave = one token, 64 / LPR of its heads (K and V). A lane holds 8
// elements: 16-byte loads, one or two words of codes.
template <typename T, int LPR, int BITS>
__global__ void __launch_bounds__(64 * KV_WAVES)
kv_write(KvCache c, KvBatch q, const T* __restrict__ k, const T* __restrict__ v, int64_t ldk, int64_t ldv, int vec,
         int32_t* __restrict__ info) {
  constexpr int W = BITS / 4;
  const int lane = threadIdx.x % 64;
  const int64_t t = int64_t(blockIdx.x) * KV_WAVES + threadIdx.x / 64;
  if (t >= q.n_tokens) return;  // whole waves; no barrier follows
  const int e = lane % LPR;
  const int h = int(blockIdx.y) * (64 / LPR) + lane / LPR;
  const bool live = h < c.heads && 8 * e < c.dim;
  float xk[8] = {}, xv[8] = {};
  if (live) {
    load8(k + t * ldk + int64_t(h) * c.dim + 8 * e, vec, xk);
    load8(v + t * ldv + int64_t(h) * c.dim + 8 * e, vec, xv);
  }
  const KvPlace p = kv_locate(c, q, t, lane, info);
  if (p.state != KV_HELD) return;
  uint32_t wk[W], wv[W];
  const uint32_t gk = quantise8<T, LPR, BITS>(xk, wk, lane);
  const uint32_t gv = quantise8<T, LPR, BITS>(xv, wv, lane);
  if (!live) return;
  const int64_t row = p.row + (int64_t(h) << c.shift);
  uint32_t* ck = c.k_codes + row * c.words + W * e;
  uint32_t* cv = c.v_codes + row * c.words + W * e;
  if constexpr (W == 1) {
    *ck = wk[0];
    *cv = wv[0];
  } else {
    *reinterpret_cast<uint2*>(ck) = uint2{wk[0], wk[1]};
    *reinterpret_cast<uint2*>(cv) = uint2{wv[0], wv[1]};
  }
  if (e == 0) {
    c.k_grid[row] = gk;
    c.v_grid[row] = gv;
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

// Same split of the work as kv_write.
template <typename T, int LPR, int BITS>
__global__ void __launch_bounds__(64 * KV_WAVES)
kv_read(KvCache c, KvBatch q, T* __restrict__ k, T* __restrict__ v, int64_t ldk, int64_t ldv, int vec,
        int32_t* __restrict__ info) {
  constexpr int W = BITS / 4;
  const int lane = threadIdx.x % 64;
  const int64_t t = int64_t(blockIdx.x) * KV_WAVES + threadIdx.x / 64;
  if (t >= q.n_tokens) return;
  const int e = lane % LPR;
  const int h = int(blockIdx.y) * (64 / LPR) + lane / LPR;
  const bool live = h < c.heads && 8 * e < c.dim;
  const KvPlace p = kv_locate(c, q, t, lane, info);
  if (p.state == KV_BEHIND || !live) return;
  float xk[8] = {}, xv[8] = {};
  if (p.state == KV_HELD) {
    const int64_t row = p.row + (int64_t(h) << c.shift);
    const uint32_t* ck = c.k_codes + row * c.words + W * e;
    const uint32_t* cv = c.v_codes + row * c.words + W * e;
    uint32_t wk[W], wv[W];
    if constexpr (W == 1) {
      wk[0] = *ck;
      wv[0] = *cv;
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(ck), b = *reinterpret_cast<const uint2*>(cv);
      wk[0] = a.x, wk[1] = a.y, wv[0] = b.x, wv[1] = b.y;
    }
    values8<BITS>(wk, c.k_grid[row], xk);
    values8<BITS>(wv, c.v_grid[row], xv);
  }
  store8(k + t * ldk + int64_t(h) * c.dim + 8 * e, vec, xk);
  store8(v + t * ldv + int64_t(h) * c.dim + 8 * e, vec, xv);
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
        using T = decltype(ty);
        const dim3 grid(unsigned((b.n_tokens + KV_WAVES - 1) / KV_WAVES),
                        unsigned((c.heads + 64 / lpr.value - 1) / (64 / lpr.value)));
        hipLaunchKernelGGL((kv_write<T, lpr.value, bits.value>), grid, dim3(64 * KV_WAVES), 0, s, c, b,
                           static_cast<const T*>(k), static_cast<const T*>(v), ldk, ldv, vec, info);
        return launch_status();
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
    return with_lanes(c.dim, [&](auto lpr) {
      return with_bits(cache->bits, [&](auto bits) {
        using T = decltype(ty);
        const dim3 grid(unsigned((b.n_tokens + KV_WAVES - 1) / KV_WAVES),
                        unsigned((c.heads + 64 / lpr.value - 1) / (64 / lpr.value)));
        hipLaunchKernelGGL((kv_read<T, lpr.value, bits.value>), grid, dim3(64 * KV_WAVES), 0, s, c, b,
                           static_cast<T*>(k), static_cast<T*>(v), ldk, ldv, vec, info);
        return launch_status();
      });
    });
  });
}
