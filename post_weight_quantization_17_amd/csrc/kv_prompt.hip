// Attention over the paged, quantised cache for calls with many query rows a
// sequence (prompts): the mathematics, operands and softmax of
// kv_attention.hip, laid out for rows instead of keys.
//
// There each wave converts the codes it multiplies with, which is free while
// the cache's bytes bound the call, but with many rows the same keys would be
// converted again for every 16 of them. Here a workgroup's 4 waves take RT
// 16-row tiles each over the same keys: 64 keys at a time are converted once,
// a quarter by each wave, and left in LDS as MFMA operands (fragments of 16
// bytes a lane, read back by lane, without bank conflicts) in two buffers: a
// barrier a tile. The codes' zeros are subtracted during the conversion, so
// both operands are the exact integers c - z. A wave skips the keys that none
// of its rows sees.
#include "kv_attention.h"

namespace gptq {
namespace {

constexpr int prompt_tiles(int dp) { return dp <= 128 ? 2 : 1; }
constexpr int prompt_waves_per_simd(int dp, bool split) { return dp == 64 || (dp == 128 && !split) ? 2 : 1; }

constexpr int ROWS_TILE = 64;  // keys at a time

template <int DP>
struct Stage {
  half8 k[4][DP / 32][64];  // [16 keys][32 d][lane]
  half8 v[2][DP / 16][64];  // [32 keys][d within a lane's share][lane]
  float sk[64], sv[64];     // scales of the keys
};

template <int BITS, int DP, bool FULL, bool SPLIT>
__global__ void __launch_bounds__(64 * ATT_WAVES, prompt_waves_per_simd(DP, SPLIT))
kv_attend_rows(AttArgs a) {
  constexpr int RT = prompt_tiles(DP), NJ = DP / 32, DPL = DP / 16;
  constexpr int KW = DP * BITS / 128;         // words of a key's quarter row
  constexpr int HB = DPL * BITS / 2;          // bits of V that a wave converts for each key and lane
  constexpr int VW = HB < 32 ? 1 : HB / 32;   // words that hold them
  constexpr uint32_t MAGIC = Half<BITS>::magic;
  constexpr int AT = Half<BITS>::at;
  __shared__ Stage<DP> stage[2];

  const KvCache& c = a.c;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int g = lane / 16, n16 = lane % 16;
  const int kv = int(blockIdx.x % unsigned(c.heads));
  const Seq sq = find_unit<false>(a, int(blockIdx.x / unsigned(c.heads)), lane);
  if (sq.b < 0) return;  // whole workgroup; uniform

  const int64_t cap = a.b.max_pages << c.shift;
  const int64_t len = sq.len;
  const int last_row = block_last_row(a, sq.n, sq.rb);
  const int nrows = last_row - sq.rb * a.block_rows + 1;
  const uint32_t kend = keys_seen(len, sq.n, last_row / a.ratio, cap);
  if (len > cap && threadIdx.x == 0) kv_flag(a.info);
  const uint32_t k0 = sq.split * sq.chunk;
  if (sq.split > 0 && k0 >= kend) return;
  const uint32_t k1 = kend - k0 < sq.chunk ? kend : k0 + sq.chunk;

  // This lane's query rows (one a tile), and the keys that all and any of the
  // tile's rows see.
  struct Row {
    int token, head, pos;
    uint32_t lim, all, any;
    float slope;
    bool live;
  };
  Row row[RT];
  Query<BITS, DP, FULL, SPLIT> q[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int first = (wave * RT + t) * 16, base = sq.rb * a.block_rows + first;
    Row& r = row[t];
    r.live = first + n16 < nrows;
    const int at = r.live ? base + n16 : 0, i = at / a.ratio;
    r.token = sq.t0 + i;
    r.head = kv * a.ratio + (at - i * a.ratio);
    r.lim = r.live ? keys_seen(len, sq.n, i, cap) : 0;
    r.pos = int(len - sq.n + i);
    const int last = first + 15 < nrows ? base + 15 : last_row;
    r.all = first < nrows ? keys_seen(len, sq.n, base / a.ratio, cap) : 0;
    r.any = first < nrows ? keys_seen(len, sq.n, last / a.ratio, cap) : 0;
    r.slope = a.slopes ? a.slopes[r.head] * LOG2E : 0.0f;
    q[t].load(a, r.live, r.token, r.head, g);
  }

  // Conversion: each wave takes 16 of the keys, and of the values the 32 keys
  // `span` and the lower or upper half of each lane's d.
  const int words = FULL ? DP * BITS / 32 : c.words;
  const int32_t* const pages = a.b.table + sq.b * a.b.ld;
  const int part = wave & 1, span = wave >> 1;
  struct Raw {
    uint32_t k[KW], v[8 * VW];
    uint32_t kg, vg;  // grids of key n16 of the wave's 16
    uint4 zg[2];      // grids of the 8 keys of the values
    uint32_t ok;      // bit u: the 16 keys u lie on a page
  };
  struct Ids {
    int id[4];
  };
  const auto look_up = [&](uint32_t p0) {
    Ids r{{-1, -1, -1, -1}};
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (p0 + 16 * u < k1) r.id[u] = pages[(p0 + 16 * u) >> c.shift];
    return r;
  };
  const int vc = n16 * DPL < c.dim ? n16 : 0;  // lanes past the head's end repeat the first one's codes
  const auto fetch = [&](uint32_t p0, const Ids& ids, Raw& raw) {
    int64_t at[4];
    raw.ok = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t p = p0 + 16 * u;
      int64_t id = __builtin_amdgcn_readfirstlane(ids.id[u]);
      if (id >= 0 && id < c.n_pages) {
        raw.ok |= 1u << u;
      } else {
        if (p < k1) kv_flag(a.info);
        id = 0;  // masked; the first page's rows are there to be read
      }
      at[u] = ((id * c.heads + kv) << c.shift) + (p & ((1u << c.shift) - 1));
    }
    const int64_t mine = wave == 0 ? at[0] : wave == 1 ? at[1] : wave == 2 ? at[2] : at[3];
    const char* kr = reinterpret_cast<const char*>(c.k_codes + mine * words);
    raw.kg = c.k_grid[mine + n16];
    raw.vg = c.v_grid[mine + n16];
    if constexpr (FULL) {
      load_words<KW>(kr + 4u * (n16 * words + g * KW), raw.k);
    } else {
      constexpr int W = BITS / 4;  // words of a block of 8 d
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int b = lane_block<DP, FULL>(g, j);
        load_words<W>(kr + 4u * (n16 * words + W * (8 * b < c.dim ? b : 0)), &raw.k[W * j]);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t base = (span ? at[2 + u] : at[u]) + 4 * g;
      raw.zg[u] = *reinterpret_cast<const uint4*>(c.v_grid + base);
      const char* vr = reinterpret_cast<const char*>(c.v_codes + base * words) + DPL * BITS / 8 * vc + HB / 8 * part;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const char* vp = vr + 4 * r * words;
        uint32_t* w = &raw.v[(4 * u + r) * VW];
        if constexpr (HB == 8)
          w[0] = *reinterpret_cast<const uint8_t*>(vp);
        else if constexpr (HB == 16)
          w[0] = *reinterpret_cast<const uint16_t*>(vp);
        else
          load_words<VW>(vp, w);
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
    const uint32_t z1 = MAGIC + (kv_zero<BITS>(raw.kg) * 0x10001u << AT);
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = z1;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      key_codes<BITS>(&raw.k[j * (BITS / 4)], h, kc);
      st.k[wave][j][lane] = minus(h, z);
    }
    if (g == 0) {
      st.sk[16 * wave + n16] = kv_scale(raw.kg);
      st.sv[16 * wave + n16] = kv_scale(raw.vg);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint4 w = raw.zg[e / 2];
      const uint32_t z0 = kv_zero<BITS>(e % 2 ? w.z : w.x), z2 = kv_zero<BITS>(e % 2 ? w.w : w.y);
      z[e] = (z0 | z2 << 16) << AT | MAGIC;
    }
    half8* out = &st.v[span][part * (DPL / 2)][lane];  // [m][lane] from this wave's first m on
#pragma unroll
    for (int vw = 0; vw < VW; ++vw) {
#pragma unroll
      for (int hi = 0; hi < (HB >= 32 ? 2 : 1); ++hi) {
        // 16 bits of this word of the keys of a pair, side by side
#pragma unroll
        for (int e = 0; e < 4; ++e)
          two[e] = __builtin_amdgcn_perm(raw.v[(2 * e + 1) * VW + vw], raw.v[2 * e * VW + vw], hi ? 0x07060302u : 0x05040100u);
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

  floatx4 o[RT][DPL];
  float M[RT], l[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    M[t] = ATT_LOWEST;
    l[t] = 0.0f;
#pragma unroll
    for (int m = 0; m < DPL; ++m) o[t][m] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // 32 of the tile's keys (half h) from p0 on; ok: bit u for its 16 keys u.
  const auto compute = [&](uint32_t p0, uint32_t ok, const Stage<DP>& st, int half) {
    floatx4 acc[RT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[t][u] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const half8 keys = st.k[2 * half + u][j][lane];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          if constexpr (SPLIT) acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(keys, q[t].l[j], acc[t][u], 0, 0, 0);
          acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(keys, q[t].h[j], acc[t][u], 0, 0, 0);
        }
      }
    }
    half8 wh[RT], wl[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const Row& r = row[t];
      float x[8], s[8];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 sk = *reinterpret_cast<const float4*>(&st.sk[32 * half + 16 * u + 4 * g]);
        const float4 sv = *reinterpret_cast<const float4*>(&st.sv[32 * half + 16 * u + 4 * g]);
        x[4 * u] = acc[t][u][0] * (sk.x * q[t].scale), x[4 * u + 1] = acc[t][u][1] * (sk.y * q[t].scale);
        x[4 * u + 2] = acc[t][u][2] * (sk.z * q[t].scale), x[4 * u + 3] = acc[t][u][3] * (sk.w * q[t].scale);
        s[4 * u] = sv.x, s[4 * u + 1] = sv.y, s[4 * u + 2] = sv.z, s[4 * u + 3] = sv.w;
      }
      if (a.slopes) {
        const float rel = float(int(p0) + 4 * g - r.pos);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(r.slope, rel + float(16 * (e / 4) + e % 4), x[e]);
      }
      if (p0 + 32 > r.all || ok != 3u) {
        const int left = int(r.lim) - int(p0) - 4 * g;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool seen = 16 * (e / 4) + e % 4 < left && (ok >> (e / 4) & 1u) != 0;
          x[e] = seen ? x[e] : -INFINITY;
          s[e] = seen ? s[e] : 0.0f;
        }
      }
      float p[8], w[8], big = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = __builtin_amdgcn_exp2f(x[e] - M[t]);
        w[e] = p[e] * s[e];
        big = fmaxf(big, w[e]);
      }
      if (__any(big > ATT_W_LIMIT)) {
        float top = ATT_LOWEST;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, x[e] + __builtin_amdgcn_logf(s[e]) - ATT_W_TOP);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        top = fmaxf(top, M[t]);
        const float f = __builtin_amdgcn_exp2f(M[t] - top);
        M[t] = top;
        l[t] *= f;
#pragma unroll
        for (int m = 0; m < DPL; ++m) o[t][m] *= f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = __builtin_amdgcn_exp2f(x[e] - M[t]);
          w[e] = p[e] * s[e];
        }
      }
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum += p[e];
        wh[t][e] = _Float16(w[e]);
        if constexpr (SPLIT) wl[t][e] = _Float16(w[e] - float(wh[t][e]));
      }
      l[t] += sum;
    }
#pragma unroll
    for (int m = 0; m < DPL; ++m) {
      const half8 values = st.v[half][m][lane];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        if constexpr (SPLIT) o[t][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(values, wl[t], o[t][m], 0, 0, 0);
        o[t][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(values, wh[t], o[t][m], 0, 0, 0);
      }
    }
  };

  // Tile n is computed from one buffer while tile n + 1 is converted into the
  // other and tile n + 2 is on its way. The barrier ends both uses.
  const uint32_t any = RT == 2 && row[RT - 1].any ? row[RT - 1].any : row[0].any;
  if (k0 < k1) {
    Raw raw;
    Ids ids = look_up(k0);
    fetch(k0, ids, raw);
    ids = look_up(k0 + ROWS_TILE);
    uint32_t ok = raw.ok;
    convert(raw, stage[0]);
    if (k0 + ROWS_TILE < k1) {
      fetch(k0 + ROWS_TILE, ids, raw);
      ids = look_up(k0 + 2 * ROWS_TILE);
    }
    __syncthreads();
    int b = 0;
    for (uint32_t p0 = k0; p0 < k1; p0 += ROWS_TILE, b ^= 1) {
      uint32_t next_ok = 0;
      if (p0 + ROWS_TILE < k1) {
        next_ok = raw.ok;
        convert(raw, stage[b ^ 1]);
        if (p0 + 2 * ROWS_TILE < k1) {
          fetch(p0 + 2 * ROWS_TILE, ids, raw);
          ids = look_up(p0 + 3 * ROWS_TILE);
        }
      }
#pragma unroll 1
      for (int h = 0; h < 2; ++h)
        if (p0 + 32 * h < any) compute(p0 + 32 * h, ok >> (2 * h) & 3u, stage[b], h);
      ok = next_ok;
      __syncthreads();
    }
  }

  // o[t][m][r] is d = (4 g + r) DPL + m of the lane's row: DPL together.
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const Row& r = row[t];
    float sum = l[t];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (!r.live) continue;
    if (kend > sq.chunk) {  // one of several
      if (sq.first + sq.split >= a.parts) continue;  // only where starts are out of order
      const int64_t pr = (int64_t(sq.first + sq.split) * c.heads + kv) * a.rows + (wave * RT + t) * 16 + n16;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = (4 * g + e) * DPL;
        if (d >= c.dim) continue;
#pragma unroll
        for (int m = 0; m < DPL; m += 4)
          *reinterpret_cast<float4*>(a.part_o + pr * c.dim + d + m) = float4{o[t][m][e], o[t][m + 1][e], o[t][m + 2][e], o[t][m + 3][e]};
      }
      if (g == 0) a.part_ml[pr] = float2{M[t], sum};
    } else {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a row that sees no key gives zeros
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = (4 * g + e) * DPL;
        if (d >= c.dim) continue;
        const int64_t at = int64_t(r.token) * a.ldo + int64_t(r.head) * c.dim + d;
        if constexpr (DPL % 8 == 0) {
#pragma unroll
          for (int m = 0; m < DPL; m += 8) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = o[t][m + k][e] * inv;
            if (a.out_dtype == GPTQ_F16)
              store8(static_cast<_Float16*>(a.out) + at + m, a.out_vec, v);
            else if (a.out_dtype == GPTQ_BF16)
              store8(static_cast<bf16*>(a.out) + at + m, a.out_vec, v);
            else
              store8(static_cast<float*>(a.out) + at + m, a.out_vec, v);
          }
        } else {
#pragma unroll
          for (int m = 0; m < DPL; ++m) store_out(a, at + m, o[t][m][e] * inv);
        }
      }
    }
  }
}

template <int BITS, int DP, bool FULL, bool SPLIT>
int launch_rows(const AttArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((kv_attend_rows<BITS, DP, FULL, SPLIT>), dim3(unsigned(a.units * a.c.heads)), dim3(64 * ATT_WAVES), 0,
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

int prompt_target(int dp, bool split) { return 256 * prompt_waves_per_simd(dp, split); }

int launch_prompt(const AttArgs& a, int bits, bool split, hipStream_t s) {
  static_assert(prompt_rows(64) == 64 * prompt_tiles(64) && prompt_rows(128) == 64 * prompt_tiles(128) &&
                    prompt_rows(256) == 64 * prompt_tiles(256),
                "a block's rows are its waves' tiles");
  return bits == 4 ? launch_rows<4>(a, split, s) : launch_rows<8>(a, split, s);
}

}  // namespace gptq
