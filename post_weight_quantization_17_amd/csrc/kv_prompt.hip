// Attention over the paged, quantised cache for calls with many query rows a
// sequence (prompts): the mathematics, operands and softmax of
// kv_attention.hip, laid out for rows instead of keys.
//
// There each wave converts the codes it multiplies with, which is free while
// the cache's bytes bound the call, but with many rows the same keys would be
// converted again for every 16 of them. Here a workgroup's 8 waves take 16
// rows each over the same keys: 64 keys at a time are converted once, an
// eighth by each wave, and left in LDS as MFMA operands (fragments of 16 bytes
// a lane, read back by lane, without bank conflicts) in two buffers: a barrier
// a tile. The codes' zeros are subtracted during the conversion, so
// both operands are the exact integers c - z. A wave skips the keys that none
// of its rows sees.
//
// Measured: two causal prompts of 1500 and 976 tokens, 32 heads over 8 of 128,
// 4 bits, 92 us with an idle join: 534 TFLOP/s over the 4.9e10 operations that
// the mask leaves (a large fp16 matrix product runs at 1137). Instructions are
// issued in 87% of the cycles (VALU 50%, scalar 19%, LDS 11%); of the 60 VALU
// operations for 32 keys of a row the 8 exponentials count fourfold. Other
// layouts of the same work: 4 waves of two row tiles 125 us, 4 waves of one
// 116, 64-row blocks whose waves halve the keys 134.
#include "kv_attention.h"

namespace gptq {
namespace {

constexpr int ROWS_WAVES = 8;
static_assert(PROMPT_BLOCK == 16 * ROWS_WAVES, "a block's rows are its waves' tiles");
// A workgroup has two waves on each SIMD; two workgroups share a CU where 128
// registers suffice.
constexpr int prompt_waves_per_simd(int dp, bool split) { return dp == 64 || (dp == 128 && !split) ? 4 : 2; }

constexpr int ROWS_TILE = 64;  // keys at a time

template <int DP>
struct Stage {
  half8 k[4][DP / 32][64];  // [16 keys][32 d][lane]
  half8 v[2][DP / 16][64];  // [32 keys][d within a lane's share][lane]
  float sk[64], sv[64];     // scales of the keys
  uint32_t ok[4];           // whether 16 keys lie on a page
};

template <int BITS, int DP, bool FULL, bool SPLIT>
__global__ void __launch_bounds__(64 * ROWS_WAVES, prompt_waves_per_simd(DP, SPLIT))
kv_attend_rows(AttArgs a) {
  constexpr int NJ = DP / 32, DPL = DP / 16;
  constexpr int KW = DP * BITS / 128;         // words of a key's quarter row
  constexpr int HB = DPL * BITS / 2;          // bits of V that a wave converts for each key and lane
  constexpr int VW = HB < 32 ? 1 : HB / 32;   // words that hold them
  constexpr uint32_t MAGIC = Half<BITS>::magic;
  constexpr int AT = Half<BITS>::at;
  __shared__ Stage<DP> stage[2];

  const KvCache& c = a.c;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int g = lane / 16, n16 = lane % 16;
  const int unit = a.by_heads(int(blockIdx.x)), kv = int(blockIdx.x) - unit * c.heads;
  const Seq sq = find_unit<false>(a, unit, lane);
  if (sq.b < 0) return;  // whole workgroup; uniform

  const int64_t cap = a.b.max_pages << c.shift;
  const int64_t len = sq.len;
  const int last_row = block_last_row(a, sq.n, sq.rb);
  const int nrows = last_row - (sq.rb << a.block_shift) + 1;
  const uint32_t kend = keys_seen(len, sq.n, a.by_ratio(last_row), cap);
  if (len > cap && threadIdx.x == 0) kv_flag(a.info);
  const uint32_t k0 = sq.split * sq.chunk;
  if (sq.split > 0 && k0 >= kend) return;
  const uint32_t k1 = kend - k0 < sq.chunk ? kend : k0 + sq.chunk;

  // This lane's query row, and the keys that all and any of the wave's rows
  // see.
  const int first = wave * 16, base_row = (sq.rb << a.block_shift) + first;
  const bool live = first + n16 < nrows;
  const int at_row = live ? base_row + n16 : 0, i = a.by_ratio(at_row);
  const int token = sq.t0 + i, head = kv * a.ratio + (at_row - i * a.ratio);
  const int pos = live ? int(len - sq.n + i) : -1;  // past no key where there is no row
  const uint32_t all = first < nrows ? keys_seen(len, sq.n, a.by_ratio(base_row), cap) : 0;
  const uint32_t any = first < nrows ? keys_seen(len, sq.n, a.by_ratio(first + 15 < nrows ? base_row + 15 : last_row), cap) : 0;
  const float slope = a.slopes ? a.slopes[head] * LOG2E : 0.0f;
  Query<BITS, DP, FULL, SPLIT> q;
  q.load(a, live, token, head, g);

  // Conversion: waves 0 to 3 take 16 of the keys each, waves 4 to 7 the values
  // of the 32 keys `span`, the lower or upper half of each lane's d.
  const int words = FULL ? DP * BITS / 32 : c.words;
  const int32_t* const pages = a.b.table + sq.b * a.b.ld;
  const int part = wave & 1, span = wave >> 1 & 1;
  struct Raw {
    uint32_t w[KW > 8 * VW ? KW : 8 * VW];
    uint4 zg[2];  // values: grids of this lane's 8 keys; keys: of key n16, of k and v
    uint32_t ok;  // keys: they lie on a page
  };
  // The pages of the keys that this wave converts: of its 16, or of the two
  // 16s of its 32 (one page if that holds them).
  const int ahead = wave < 4 ? 16 * wave : 32 * span;
  const bool one_page = wave < 4 || c.shift >= 5;
  struct Ids {
    int id[2];
  };
  const auto look_up = [&](uint32_t p0) {
    Ids r{{-1, -1}};
    const uint32_t p = p0 + ahead;
    if (p < k1) r.id[0] = pages[p >> c.shift];
    if (!one_page && p + 16 < k1) r.id[1] = pages[(p + 16) >> c.shift];
    return r;
  };
  const int vc = n16 * DPL < c.dim ? n16 : 0;  // lanes past the head's end repeat the first one's codes
  uint32_t v_off = 16u * g * words + DPL * BITS / 8 * vc + HB / 8 * part;
  uint32_t k_off = FULL ? 4u * (n16 * words + g * KW) : 4u * n16 * words;
  uint32_t key_off = 4u * n16, quad_off = 16u * g;  // of grid words
  const auto fetch = [&](uint32_t p0, const Ids& ids, Raw& raw) {
    const uint32_t p = p0 + ahead;
    const Place16 first = place16(c, a.info, kv, ids.id[0], p, k1);
    raw.ok = first.ok;
    // Base pointers are uniform, offsets 32 bits a lane; their sums are formed
    // by the loads.
    KV_FRESH_V(v_off);
    KV_FRESH_V(k_off);
    KV_FRESH_V(key_off);
    KV_FRESH_V(quad_off);
    if (wave < 4) {
      const char* kr = reinterpret_cast<const char*>(c.k_codes) + first.codes;
      raw.zg[0].x = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const char*>(c.k_grid) + first.grid + key_off);
      raw.zg[0].y = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const char*>(c.v_grid) + first.grid + key_off);
      if constexpr (FULL) {
        load_words<KW>(kr + k_off, raw.w);
      } else {
        constexpr int W = BITS / 4;  // words of a block of 8 d
        uint32_t fresh_g = g;        // the blocks' offsets are formed here, not kept
        KV_FRESH_V(fresh_g);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int b = lane_block<DP, FULL>(int(fresh_g), j);
          load_words<W>(kr + (k_off + 4u * W * (8 * b < c.dim ? b : 0)), &raw.w[W * j]);
        }
      }
    } else {
      const Place16 second = one_page ? first.next(words) : place16(c, a.info, kv, ids.id[1], p + 16, k1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const Place16& at = u ? second : first;
        raw.zg[u] = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(c.v_grid) + at.grid + quad_off);
        const char* vr = reinterpret_cast<const char*>(c.v_codes) + at.codes;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const char* vp = vr + 4 * r * words + v_off;
          uint32_t* w = &raw.w[(4 * u + r) * VW];
          if constexpr (HB == 8)
            w[0] = *reinterpret_cast<const uint8_t*>(vp);
          else if constexpr (HB == 16)
            w[0] = *reinterpret_cast<const uint16_t*>(vp);
          else
            load_words<VW>(vp, w);
        }
      }
    }
  };
  const Consts kc = conversion_consts<BITS>();
  const auto minus = [](const uint32_t (&h)[4], const uint32_t (&z)[4]) {
    uint32_t s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = as_u32(as_half2(h[e]) - as_half2(z[e]));
    return as_half8(s[0], s[1], s[2], s[3]);
  };
  const auto convert = [&](const Raw& raw, Stage<DP>& st) {
    uint32_t h[4], z[4], two[4];
    if (wave < 4) {
      const uint32_t z1 = MAGIC + (kv_zero<BITS>(raw.zg[0].x) * 0x10001u << AT);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = z1;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        key_codes<BITS>(&raw.w[j * (BITS / 4)], h, kc);
        st.k[wave][j][lane] = minus(h, z);
      }
      if (g == 0) {
        st.sk[16 * wave + n16] = kv_scale(raw.zg[0].x);
        st.sv[16 * wave + n16] = kv_scale(raw.zg[0].y);
        st.ok[wave] = raw.ok;
      }
      return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint4 w = raw.zg[e / 2];
      const uint32_t z0 = kv_zero<BITS>(e % 2 ? w.z : w.x), z1 = kv_zero<BITS>(e % 2 ? w.w : w.y);
      z[e] = (z0 | z1 << 16) << AT | MAGIC;
    }
    half8* out = &st.v[span][part * (DPL / 2)][lane];  // [m][lane] from this wave's first m on
#pragma unroll
    for (int vw = 0; vw < VW; ++vw) {
#pragma unroll
      for (int hi = 0; hi < (HB >= 32 ? 2 : 1); ++hi) {
        // 16 bits of this word of the keys of a pair, side by side
#pragma unroll
        for (int e = 0; e < 4; ++e)
          two[e] = __builtin_amdgcn_perm(raw.w[(2 * e + 1) * VW + vw], raw.w[2 * e * VW + vw], hi ? 0x07060302u : 0x05040100u);
        constexpr int PER = 16 / BITS < DPL / 2 ? 16 / BITS : DPL / 2;  // d in them
        half8* o = out + 64 * ((2 * vw + hi) * (16 / BITS));
#pragma unroll
        for (int m = 0; m < PER; ++m) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (BITS == 4)
              h[e] = m == 0 ? nibbles<0>(two[e], kc) : m == 1 ? nibbles<1>(two[e], kc) : m == 2 ? nibbles<2>(two[e], kc)
                                                                                                 : nibbles<3>(two[e], kc);
            else
              h[e] = m == 0 ? byte_pair<0, 2>(two[e], kc) : byte_pair<1, 3>(two[e], kc);
          }
          o[64 * m] = minus(h, z);
        }
      }
    }
  };

  floatx4 o[DPL];
  float M = ATT_LOWEST, l = 0.0f;
#pragma unroll
  for (int m = 0; m < DPL; ++m) o[m] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  // 32 of the tile's keys (half h) from p0 on.
  const auto compute = [&](uint32_t p0, const Stage<DP>& st, int half) {
    const uint32_t ok = __builtin_amdgcn_readfirstlane(st.ok[2 * half] | st.ok[2 * half + 1] << 1);
    float x[8], s[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const half8 keys = st.k[2 * half + u][j][lane];
        if constexpr (SPLIT) acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(keys, q.l[j], acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(keys, q.h[j], acc, 0, 0, 0);
      }
      const float4 sk = *reinterpret_cast<const float4*>(&st.sk[32 * half + 16 * u + 4 * g]);
      const float4 sv = *reinterpret_cast<const float4*>(&st.sv[32 * half + 16 * u + 4 * g]);
      x[4 * u] = acc[0] * (sk.x * q.scale), x[4 * u + 1] = acc[1] * (sk.y * q.scale);
      x[4 * u + 2] = acc[2] * (sk.z * q.scale), x[4 * u + 3] = acc[3] * (sk.w * q.scale);
      s[4 * u] = sv.x, s[4 * u + 1] = sv.y, s[4 * u + 2] = sv.z, s[4 * u + 3] = sv.w;
    }
    if (a.slopes) {
      const float rel = float(int(p0) + 4 * g - pos);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(slope, rel + float(16 * (e / 4) + e % 4), x[e]);
    }
    if (p0 + 32 > all || ok != 3u) {
      const int seen_to = pos < int(k1) ? pos + 1 : int(k1);
      const int left = seen_to - int(p0) - 4 * g;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool seen = 16 * (e / 4) + e % 4 < left && (ok >> (e / 4) & 1u) != 0;
        x[e] = seen ? x[e] : -INFINITY;
        s[e] = seen ? s[e] : 0.0f;
      }
    }
    float w[8], sum = 0.0f, big = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = __builtin_amdgcn_exp2f(x[e] - M);
      sum += p;
      w[e] = p * s[e];
      big = fmaxf(big, w[e]);
    }
    if (__any(big > ATT_W_LIMIT || sum > ATT_SUM_LIMIT)) {
      float top = ATT_LOWEST;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, x[e] + fmaxf(__builtin_amdgcn_logf(s[e]), ATT_S_LEAST) - ATT_W_TOP);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      top = fmaxf(top, M);
      const float f = __builtin_amdgcn_exp2f(M - top);
      M = top;
      l *= f;
#pragma unroll
      for (int m = 0; m < DPL; ++m) o[m] *= f;
      sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = __builtin_amdgcn_exp2f(x[e] - M);
        sum += p;
        w[e] = p * s[e];
      }
    }
    l += sum;
    half8 wh, wl;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      wh[e] = _Float16(w[e]);
      if constexpr (SPLIT) wl[e] = _Float16(w[e] - float(wh[e]));
    }
#pragma unroll
    for (int m = 0; m < DPL; ++m) {
      const half8 values = st.v[half][m][lane];
      if constexpr (SPLIT) o[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(values, wl, o[m], 0, 0, 0);
      o[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(values, wh, o[m], 0, 0, 0);
    }
  };

  // Tile n is computed from one buffer while tile n + 1 is converted into the
  // other and tile n + 2 is on its way. The barrier ends both uses.
  if (k0 < k1) {
    Raw raw;
    Ids ids = look_up(k0);
    fetch(k0, ids, raw);
    ids = look_up(k0 + ROWS_TILE);
    convert(raw, stage[0]);
    if (k0 + ROWS_TILE < k1) {
      fetch(k0 + ROWS_TILE, ids, raw);
      ids = look_up(k0 + 2 * ROWS_TILE);
    }
    __syncthreads();
    int b = 0;
    for (uint32_t p0 = k0; p0 < k1; p0 += ROWS_TILE, b ^= 1) {
      if (p0 + ROWS_TILE < k1) {
        convert(raw, stage[b ^ 1]);
        if (p0 + 2 * ROWS_TILE < k1) {
          fetch(p0 + 2 * ROWS_TILE, ids, raw);
          ids = look_up(p0 + 3 * ROWS_TILE);
        }
      }
#pragma unroll 1
      for (int h = 0; h < 2; ++h)
        if (p0 + 32 * h < any) compute(p0 + 32 * h, stage[b], h);
      __syncthreads();
    }
  }

  // o[m][r] is d = (4 g + r) DPL + m of the lane's row: DPL together.
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (!live) return;
  if (kend > sq.chunk) {  // one of several
    if (sq.first + sq.split >= a.parts) return;  // only where starts are out of order
    const int64_t pr = (int64_t(sq.first + sq.split) * c.heads + kv) * a.rows + first + n16;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = (4 * g + e) * DPL;
      if (d >= c.dim) continue;
#pragma unroll
      for (int m = 0; m < DPL; m += 4)
        *reinterpret_cast<float4*>(a.part_o + pr * c.dim + d + m) = float4{o[m][e], o[m + 1][e], o[m + 2][e], o[m + 3][e]};
    }
    if (g == 0) a.part_ml[pr] = float2{M, l};
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that sees no key gives zeros
  // The row's place is worked out again rather than kept through the loop.
  uint32_t out_row = uint32_t(base_row + n16);
  KV_OPAQUE_V(out_row);
  const int out_i = a.by_ratio(int(out_row));
  const int64_t out_at = int64_t(sq.t0 + out_i) * a.ldo + int64_t(kv * a.ratio + (int(out_row) - out_i * a.ratio)) * c.dim;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int d = (4 * g + e) * DPL;
    if (d >= c.dim) continue;
    const int64_t at = out_at + d;
    if constexpr (DPL % 8 == 0) {
#pragma unroll
      for (int m = 0; m < DPL; m += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = o[m + k][e] * inv;
        if (a.out_dtype == GPTQ_F16)
          store8(static_cast<_Float16*>(a.out) + at + m, a.out_vec, v);
        else if (a.out_dtype == GPTQ_BF16)
          store8(static_cast<bf16*>(a.out) + at + m, a.out_vec, v);
        else
          store8(static_cast<float*>(a.out) + at + m, a.out_vec, v);
      }
    } else {
#pragma unroll
      for (int m = 0; m < DPL; ++m) store_out(a, at + m, o[m][e] * inv);
    }
  }
}

template <int BITS, int DP, bool FULL, bool SPLIT>
int launch_rows(const AttArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((kv_attend_rows<BITS, DP, FULL, SPLIT>), dim3(unsigned(a.units * a.c.heads)), dim3(64 * ROWS_WAVES), 0,
                     s, a);
  return launch_status();
}
template <int BITS, int DP>
int launch_rows(const AttArgs& a, bool split, hipStream_t s) {
  if (a.c.dim == DP) return split ? launch_rows<BITS, DP, true, true>(a, s) : launch_rows<BITS, DP, true, false>(a, s);
  return split ? launch_rows<BITS, DP, false, true>(a, s) : launch_rows<BITS, DP, false, false>(a, s);
}
template <int BITS>
int launch_rows(const AttArgs& a, bool split, hipStream_t s) {
  if (a.c.dim <= 64) return launch_rows<BITS, 64>(a, split, s);
  if (a.c.dim <= 128) return launch_rows<BITS, 128>(a, split, s);
  return launch_rows<BITS, 256>(a, split, s);
}

}  // namespace

int launch_prompt(const AttArgs& a, int bits, bool split, hipStream_t s) {
  return bits == 4 ? launch_rows<4>(a, split, s) : launch_rows<8>(a, split, s);
}

}  // namespace gptq
