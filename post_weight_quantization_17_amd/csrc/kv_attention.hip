// Attention of new tokens over the paged, quantised key-value cache.
//
//   out[t][h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j + slope_h (j - pos_t)),  j <= pos_t
//   k_j = s (c - z) per token and head (astro-blog survey, section 1.2), v_j likewise.
//
// Rows. The query rows of one sequence and key-value head (its new tokens
// times the query heads that share the head) are taken 16 at a time: a
// 16-row block is one side of v_mfma_f32_16x16x32_f16, the keys or the head
// dimension the other. With fewer rows (a head of its own, one token) the
// spare columns cost matrix-core time that is free here, since the product
// is bound by the cache's bytes and by their conversion. Calls with very many
// rows go to the prompts' kernel (kv_prompt.hip).
//
// Operands. The codes enter the MFMAs as integers: a 4-bit code c, moved to
// bits 4..7 of an fp16 half and OR-ed under the exponent of 64, is 64 + c
// exactly (bits 6..9 and 16 + c would take a fourth shift a word); an 8-bit
// one under the exponent of 1024 is 1024 + c. Scales and zeros stay outside:
//   S[key][row] = s_k (sum_d (off + c) q - (off + z_k) sum_d q)   (fp32)
//   O[d][row]   = sum_key (c - z_v) w,  w = p s_v                 (c - z exact in fp16)
// No step rounds a dequantised value. The scores leave the first product
// with lane = row, 4 keys a lane (C/D layout); the second takes its B
// operand with lane = row, 8 keys a lane, and the order of the keys within
// an MFMA is free as long as both operands agree. So two 16-key score tiles
// are the second product's operand as they lie: no transposition, no LDS. V
// is transposed in registers: a lane loads the same few codes of its 8 keys
// and pairs the codes of two keys of one d in the halves of a word.
//
// Softmax. One running reference M per row, in log2 units, for both sums:
// w = 2^(x - M) s_v goes to fp16, l = sum 2^(x - M) stays fp32. M is chosen so
// that the largest w is 2^8 and moves only when some w passes 2^15, which
// keeps w at full fp16 precision from 2^-22 of the largest on and lets most
// tiles skip the rescaling. Steps of v below 2^-96 count as 2^-96 there, since
// the weights without them, 2^8 / s_v, would leave fp32; l stays below 2^127 for
// 2^22 keys of such weights. Queries are scaled to a largest element of 2^13
// to 2^14, exact for 16-bit types (bf16's exponents do not fit fp16); the
// power of two is put back in fp32. fp32 queries, and weights for fp32
// outputs, are split into two fp16 parts, each with its own MFMA.
//
// Split. A workgroup's 4 waves take 32-key tiles in turn and are joined
// through LDS; where the rows alone do not fill the GPU, a row block's keys
// are split over workgroups too (Seq in kv_attention.h), whose partial sums
// kv_join adds in a fixed order. Each partial result has its M; all
// reductions are fp32.
//
// Measured (one MI355X, whose large copy runs at 5.1 TB/s): 24 sequences of
// 2048 tokens, 96 heads of 128, 4 bits: 127 us, 5.1 TB/s of codes and grids;
// there the VALU is 67% busy with 340 instructions a tile (64 conversions for
// the keys, 96 for the values, 100 for the softmax). 64 ragged sequences of up
// to 8192 tokens, 8 heads, 8 bits: 73 us (3.7 TB/s). One of 131072 tokens, 8
// heads for 64, 4 bits: 41 us (3.5 TB/s): 35 us here, against 28 for the bytes
// alone (the chain length -> page -> codes and the tail), then the join. One short
// sequence, replayed in a graph: 5.5 us up to 128 tokens, 6.9 up to 256. Two tiles in flight a wave
// (at 2 waves a SIMD instead of 3) were slower, 144 against 136 us on the first.
#include "kv_attention.h"

namespace gptq {
namespace {

// Waves that share a SIMD: as many as the registers of a form leave without
// spilling (a tile in flight and one in work, the sums of DP / 16 MFMAs).
constexpr int att_waves_per_simd(int bits, int dp, bool split) {
  return dp == 256 ? (bits == 8 && split ? 1 : 2) : dp == 128 ? (bits == 8 && split ? 2 : 3) : (split ? 3 : 4);
}

// A lane's share of one 32-key tile, as loaded.
template <int BITS, int DP>
struct Tile {
  static constexpr int KW = DP * BITS / 128;          // words of a key's quarter row
  static constexpr int DPL = DP / 16;                 // d of a lane in V
  static constexpr int VW = (DPL * BITS + 31) / 32;   // words that hold them
  uint32_t k[2][KW];
  uint32_t v[8][VW];
  uint4 kg[2], vg[2];
  uint32_t kz[2];
};

template <int BITS, int DP, bool FULL, bool SPLIT>
__global__ void __launch_bounds__(64 * ATT_WAVES, att_waves_per_simd(BITS, DP, SPLIT))
kv_attend(AttArgs a) {
  using TL = Tile<BITS, DP>;
  constexpr int NJ = DP / 32, KW = TL::KW, DPL = TL::DPL, VW = TL::VW;
  constexpr float OFF = Half<BITS>::off;
  constexpr uint32_t MAGIC = Half<BITS>::magic;
  __shared__ float lds_o[2][ATT_ROWS][DP];
  __shared__ float lds_m[ATT_WAVES][ATT_ROWS], lds_l[ATT_WAVES][ATT_ROWS];

  const KvCache& c = a.c;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int g = lane / 16, n16 = lane % 16;
  const int unit = a.by_heads(int(blockIdx.x)), kv = int(blockIdx.x) - unit * c.heads;
  // A tile's pages are the table entries of its two 16-key subtiles.
  struct Ids {
    int id[2];
  };
  Ids ids{{-1, -1}};
  Seq sq;
  const bool plain = !a.splits && !a.b.starts;  // one unit a row block, one token a sequence
  if (plain) {
    // The first tile's pages are known without the length: both loads at once.
    const int b = a.per_token == 1 ? unit : unit / a.per_token;
    sq = Seq{b, b, 1, unit - b * a.per_token, 0, 1, 0, 0, 0xFFFFFF80u};
    const int len_now = a.b.lens[sq.b];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int page = (wave * ATT_TILE + 16 * u) >> c.shift;
      if (page < a.b.max_pages) ids.id[u] = a.b.table[sq.b * a.b.ld + page];
    }
    sq.len = __builtin_amdgcn_readfirstlane(len_now);
  } else {
    sq = find_unit<false>(a, unit, lane);
    if (sq.b < 0) return;  // whole workgroup; uniform
  }

  const int64_t cap = a.b.max_pages << c.shift;
  const int64_t len = sq.len;
  const int last_row = block_last_row(a, sq.n, sq.rb);
  const int nrows = last_row - sq.rb * ATT_ROWS + 1;
  const uint32_t kend = keys_seen(len, sq.n, a.by_ratio(last_row), cap);
  if (len > cap && threadIdx.x == 0) kv_flag(a.info);
  const uint32_t k0 = sq.split * sq.chunk;
  if (sq.split > 0 && k0 >= kend) return;
  const uint32_t k1 = kend - k0 < sq.chunk ? kend : k0 + sq.chunk;

  // This lane's query row, and the keys that every row of the block sees.
  const int row = sq.rb * ATT_ROWS + n16;
  const bool live = n16 < nrows;
  const int i = live ? a.by_ratio(row) : 0;
  const int hq = kv * a.ratio + (live ? row - i * a.ratio : 0);
  const uint32_t lim = live ? keys_seen(len, sq.n, i, cap) : 0;
  const uint32_t all_see = keys_seen(len, sq.n, a.by_ratio(sq.rb * ATT_ROWS), cap);
  const int pos = int(len - sq.n + i);
  const float slope = a.slopes ? a.slopes[hq] * LOG2E : 0.0f;

  // The tiles of this wave. A tile's pages are looked up a tile ahead, its
  // keys are loaded while the tile before is in its softmax and second
  // product, its values while it is in its own first product: the registers
  // of one tile suffice, and loads are always in flight.
  constexpr uint32_t step = ATT_WAVES * ATT_TILE;
  const int words = FULL ? DP * BITS / 32 : c.words;
  const int32_t* const pages = a.b.table + sq.b * a.b.ld;
  const bool one_page = c.shift >= 5;  // a tile's keys lie on one page
  const auto look_up = [&](uint32_t p0) {
    Ids r{{-1, -1}};
    if (p0 < k1) r.id[0] = pages[p0 >> c.shift];
    if (!one_page && p0 + 16 < k1) r.id[1] = pages[(p0 + 16) >> c.shift];
    return r;
  };
  struct Rows {
    Place16 u[2];
  };
  const auto locate = [&](uint32_t p0, const Ids& ids) {
    Rows r;
    r.u[0] = place16(c, a.info, kv, ids.id[0], p0, k1);
    r.u[1] = one_page ? r.u[0].next(words) : place16(c, a.info, kv, ids.id[1], p0 + 16, k1);
    return r;
  };
  const int vc = n16 * DPL < c.dim ? n16 : 0;  // lanes past the head's end repeat the first one's codes
  uint32_t k_off = FULL ? 4u * (n16 * words + g * KW) : 4u * n16 * words;
  uint32_t key_off = 4u * n16, quad_off = 16u * g;  // of grid words
  uint32_t v_off = DPL * BITS == 16 ? 16u * g * words + 2u * vc : 16u * g * words + 4u * VW * vc;
  const auto blk = [&](int j) { return lane_block<DP, FULL>(g, j); };
  TL t;
  // Base pointers are uniform, offsets 32 bits a lane; their sums are formed by
  // the loads.
  const auto load_keys = [&](const Rows& at) {
    KV_FRESH_V(k_off);
    KV_FRESH_V(key_off);
    KV_FRESH_V(quad_off);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const char* kr = reinterpret_cast<const char*>(c.k_codes) + at.u[u].codes;
      const char* gr = reinterpret_cast<const char*>(c.k_grid) + at.u[u].grid;
      if constexpr (FULL) {
        load_words<KW>(kr + k_off, t.k[u]);
      } else {
        constexpr int W = BITS / 4;  // words of a block
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          load_words<W>(kr + (k_off + 4u * W * (8 * blk(j) < c.dim ? blk(j) : 0)), &t.k[u][W * j]);
      }
      t.kg[u] = *reinterpret_cast<const uint4*>(gr + quad_off);
      if constexpr (SPLIT) t.kz[u] = *reinterpret_cast<const uint32_t*>(gr + key_off);
    }
  };
  const auto load_values = [&](const Rows& at) {
    KV_FRESH_V(v_off);
    KV_FRESH_V(quad_off);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      t.vg[u] = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(c.v_grid) + at.u[u].grid + quad_off);
      const char* vr = reinterpret_cast<const char*>(c.v_codes) + at.u[u].codes;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const char* vp = vr + 4 * r * words + v_off;
        if constexpr (DPL * BITS == 16)
          t.v[4 * u + r][0] = *reinterpret_cast<const uint16_t*>(vp);
        else
          load_words<VW>(vp, t.v[4 * u + r]);
      }
    }
  };

  uint32_t p0 = k0 + wave * ATT_TILE;
  Rows at = {};
  if (!plain) ids = look_up(p0);
  if (p0 < k1) {
    at = locate(p0, ids);
    load_keys(at);
    load_values(at);
    ids = look_up(p0 + step);
  }

  Query<BITS, DP, FULL, SPLIT> q;
  q.load(a, live, sq.t0 + i, hq, g);

  floatx4 o[DPL];
#pragma unroll
  for (int m = 0; m < DPL; ++m) o[m] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  float M = ATT_LOWEST, l = 0.0f;
  const Consts kc = conversion_consts<BITS>();

  while (p0 < k1) {
    const uint32_t ok = at.u[0].ok | at.u[1].ok << 1;
    const bool more = p0 + step < k1;
    float x[8], sv[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint32_t h[4];
        key_codes<BITS>(&t.k[u][j * (BITS / 4)], h, kc);
        if constexpr (SPLIT) {
          const uint32_t z1 = MAGIC + (kv_zero<BITS>(t.kz[u]) * 0x10001u << Half<BITS>::at);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = as_u32(as_half2(h[e]) - as_half2(z1));
        }
        const half8 keys = as_half8(h[0], h[1], h[2], h[3]);
        if constexpr (SPLIT) acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(keys, q.l[j], acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(keys, q.h[j], acc, 0, 0, 0);
      }
      const uint32_t kg[4] = {t.kg[u].x, t.kg[u].y, t.kg[u].z, t.kg[u].w};
      const uint32_t vg[4] = {t.vg[u].x, t.vg[u].y, t.vg[u].z, t.vg[u].w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float s = kv_scale(kg[r]) * q.scale;
        x[4 * u + r] = SPLIT ? acc[r] * s : fmaf(-(OFF + float(kv_zero<BITS>(kg[r]))), q.sum, acc[r]) * s;
        sv[4 * u + r] = kv_scale(vg[r]);
      }
    }
    if (more) {
      at = locate(p0 + step, ids);
      load_keys(at);
      ids = look_up(p0 + 2 * step);
    }
    if (a.slopes) {
      const float rel = float(int(p0) + 4 * g - pos);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(slope, rel + float(16 * (e / 4) + e % 4), x[e]);
    }
    if (p0 + ATT_TILE > all_see || ok != 3u) {
      const int left = int(lim) - int(p0) - 4 * g;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool seen = 16 * (e / 4) + e % 4 < left && (ok >> (e / 4) & 1u) != 0;
        x[e] = seen ? x[e] : -INFINITY;
        sv[e] = seen ? sv[e] : 0.0f;
      }
    }
    float w[8], sum = 0.0f, big = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = __builtin_amdgcn_exp2f(x[e] - M);
      sum += p;
      w[e] = p * sv[e];
      big = fmaxf(big, w[e]);
    }
    if (__any(big > ATT_W_LIMIT || sum > ATT_SUM_LIMIT)) {
      float top = ATT_LOWEST;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, x[e] + fmaxf(__builtin_amdgcn_logf(sv[e]), ATT_S_LEAST) - ATT_W_TOP);
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
        w[e] = p * sv[e];
      }
    }
    l += sum;
    half8 wh, wl;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      wh[e] = _Float16(w[e]);
      if constexpr (SPLIT) wl[e] = _Float16(w[e] - float(wh[e]));
    }
    // off + z of key pairs 2e, 2e + 1, as halves.
    uint32_t zp[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint4 w = t.vg[e / 2];
      const uint32_t z0 = kv_zero<BITS>(e % 2 ? w.z : w.x), z1 = kv_zero<BITS>(e % 2 ? w.w : w.y);
      zp[e] = (z0 | z1 << 16) << Half<BITS>::at | MAGIC;
    }
    const auto product = [&](int m, const uint32_t (&h)[4]) {
      uint32_t s[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = as_u32(as_half2(h[e]) - as_half2(zp[e]));
      const half8 vcodes = as_half8(s[0], s[1], s[2], s[3]);
      if constexpr (SPLIT) o[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vcodes, wl, o[m], 0, 0, 0);
      o[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vcodes, wh, o[m], 0, 0, 0);
    };
#pragma unroll
    for (int vw = 0; vw < VW; ++vw) {
      // Low and high 16 bits of this word of the keys of a pair, side by side.
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo[e] = __builtin_amdgcn_perm(t.v[2 * e + 1][vw], t.v[2 * e][vw], 0x05040100u);
        hi[e] = __builtin_amdgcn_perm(t.v[2 * e + 1][vw], t.v[2 * e][vw], 0x07060302u);
      }
      uint32_t h[4];
      if constexpr (BITS == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = nibbles<0>(lo[e], kc);
        product(8 * vw + 0, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = nibbles<1>(lo[e], kc);
        product(8 * vw + 1, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = nibbles<2>(lo[e], kc);
        product(8 * vw + 2, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = nibbles<3>(lo[e], kc);
        product(8 * vw + 3, h);
        if constexpr (DPL > 4) {
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = nibbles<0>(hi[e], kc);
          product(8 * vw + 4, h);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = nibbles<1>(hi[e], kc);
          product(8 * vw + 5, h);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = nibbles<2>(hi[e], kc);
          product(8 * vw + 6, h);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = nibbles<3>(hi[e], kc);
          product(8 * vw + 7, h);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = byte_pair<0, 2>(lo[e], kc);
        product(4 * vw + 0, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = byte_pair<1, 3>(lo[e], kc);
        product(4 * vw + 1, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = byte_pair<0, 2>(hi[e], kc);
        product(4 * vw + 2, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = byte_pair<1, 3>(hi[e], kc);
        product(4 * vw + 3, h);
      }
    }
    if (more) load_values(at);
    p0 += step;
  }

  // Join the waves: waves 0 and 1 leave their sums, waves 2 and 3 add theirs.
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) {
    lds_m[wave][n16] = M;
    lds_l[wave][n16] = l;
  }
  __syncthreads();
  float Mt = lds_m[0][n16];
#pragma unroll
  for (int w = 1; w < ATT_WAVES; ++w) Mt = fmaxf(Mt, lds_m[w][n16]);
  const float f = __builtin_amdgcn_exp2f(M - Mt);
  float* mine = &lds_o[wave % 2][n16][4 * g * DPL];  // o[m][r] is d = (4 g + r) DPL + m
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (wave / 2 == half && live) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int m = 0; m < DPL; ++m) {
          const float v = o[m][r] * f;
          if (half == 0)
            mine[r * DPL + m] = v;
          else
            mine[r * DPL + m] += v;
        }
    }
    __syncthreads();
  }
  for (int r = wave; r < nrows; r += ATT_WAVES) {
    const int at = sq.rb * ATT_ROWS + r;
    const int tok = a.by_ratio(at);
    const int64_t t = sq.t0 + tok;
    const int h = kv * a.ratio + (at - tok * a.ratio);
    float top = lds_m[0][r];
    for (int w = 1; w < ATT_WAVES; ++w) top = fmaxf(top, lds_m[w][r]);
    float sum = 0.0f;
    for (int w = 0; w < ATT_WAVES; ++w) sum += lds_l[w][r] * __builtin_amdgcn_exp2f(lds_m[w][r] - top);
    if (kend > sq.chunk) {  // one of several
      if (sq.first + sq.split >= a.parts) break;  // only where starts are out of order
      const int64_t pr = (int64_t(sq.first + sq.split) * c.heads + kv) * a.rows + r;
      for (int d = lane; d < c.dim; d += 64)
        a.part_o[pr * c.dim + d] = lds_o[0][r][d] + lds_o[1][r][d];
      if (lane == 0) a.part_ml[pr] = float2{top, sum};
    } else {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a row that sees no key gives zeros
      for (int d = lane; d < c.dim; d += 64) {
        const float v = (lds_o[0][r][d] + lds_o[1][r][d]) * inv;
        store_out(a, t * a.ldo + int64_t(h) * c.dim + d, v);
      }
    }
  }
}

// Joins the units of a row block's rows, in a fixed order: `rows` workgroups
// share them. Every thread holds 4 of a row's d for one residue of the units
// (lanes of a power of two cover the row), so 4 to 64 units are read at a
// time, each thread rescaling its own sum as it goes; then the residues' sums
// are added in order.
__global__ void __launch_bounds__(64 * ATT_WAVES)
kv_join(AttArgs a, int rows) {
  __shared__ float4 sums[64 * ATT_WAVES];
  __shared__ float tops[64], weights[64];
  const KvCache& c = a.c;
  const int lane = threadIdx.x % 64;
  const int pair = int(blockIdx.x / unsigned(rows)), block = a.by_heads(pair), kv = pair - block * c.heads;
  const Seq sq = find_unit<true>(a, block, lane);
  if (sq.b < 0) return;
  const int last_row = block_last_row(a, sq.n, sq.rb);
  const uint32_t kend = keys_seen(sq.len, sq.n, a.by_ratio(last_row), a.b.max_pages << c.shift);
  if (kend <= sq.chunk) return;  // kv_attend wrote the rows
  const int active = int((kend - 1) / sq.chunk) + 1;
  if (sq.first + active > a.parts) return;  // only where starts are out of order
  const int64_t stride = int64_t(c.heads) * a.rows;
  const int quads = c.dim / 4;
  const int per = quads <= 4 ? 4 : quads <= 8 ? 8 : quads <= 16 ? 16 : quads <= 32 ? 32 : 64;
  const int d4 = int(threadIdx.x) % per, residue = int(threadIdx.x) / per, residues = 64 * ATT_WAVES / per;

  for (int r = int(blockIdx.x) - pair * rows; r <= last_row - (sq.rb << a.block_shift); r += rows) {
    const int64_t pr = (int64_t(sq.first) * c.heads + kv) * a.rows + r;
    const int row = (sq.rb << a.block_shift) + r, tok = a.by_ratio(row);
    const int64_t t = sq.t0 + tok;
    const int h = kv * a.ratio + (row - tok * a.ratio);
    float4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    float top = ATT_LOWEST, sum = 0.0f;
    const float4* src = reinterpret_cast<const float4*>(a.part_o) + pr * quads + (d4 < quads ? d4 : 0);
#pragma unroll 4
    for (int s = residue; s < active; s += residues) {
      const float4 v = src[s * stride * quads];
      const float2 ml = a.part_ml[s * stride + pr];
      const float m = fmaxf(top, ml.x);
      const float f0 = __builtin_amdgcn_exp2f(top - m), f1 = __builtin_amdgcn_exp2f(ml.x - m);
      top = m;
      sum = fmaf(ml.y, f1, sum * f0);
      o.x = fmaf(v.x, f1, o.x * f0);
      o.y = fmaf(v.y, f1, o.y * f0);
      o.z = fmaf(v.z, f1, o.z * f0);
      o.w = fmaf(v.w, f1, o.w * f0);
    }
    sums[threadIdx.x] = o;
    if (d4 == 0) {
      tops[residue] = top;
      weights[residue] = sum;
    }
    __syncthreads();
    const int d = int(threadIdx.x);
    if (d < c.dim) {
      const float* flat = reinterpret_cast<const float*>(sums);
      const int used = active < residues ? active : residues;
      top = tops[0];
      for (int i = 1; i < used; ++i) top = fmaxf(top, tops[i]);
      float v = 0.0f;
      sum = 0.0f;
      for (int i = 0; i < used; ++i) {
        const float f = __builtin_amdgcn_exp2f(tops[i] - top);
        v = fmaf(flat[i * per * 4 + d], f, v);
        sum = fmaf(weights[i], f, sum);
      }
      v *= sum == 0.0f ? 0.0f : 1.0f / sum;
      store_out(a, t * a.ldo + int64_t(h) * c.dim + d, v);
    }
    __syncthreads();  // the next row overwrites the sums
  }
}

constexpr int64_t JOIN_GROUPS = 1024;  // workgroups of a join, or one a row block if those are more

// Least query rows (over all heads) of a call for the prompts' kernel, which
// also asks for a whole row block a sequence in the mean. It converts the cache
// once for 128 rows, but needs many row blocks to fill the GPU and to balance
// the causal mask. Measured (us, prompts' kernel and the other; 2000 cached
// tokens; rows are tokens times query heads):
//   8 sequences, 32 heads over 8, 4 bits:  32768 rows  98 / 104, 65536 rows 114 / 196
//   8 sequences, 32 heads, 8 bits:         32768 rows 142 / 129, 49152 rows 138 / 183
//   1 sequence, 32 heads over 8, 4 bits:    8192 rows  52 /  58,  4096 rows  39 /  34
constexpr int64_t PROMPT_MIN_ROWS = 384 * PROMPT_BLOCK;

// How a call is cut: everything that does not depend on device data, nor on
// the types (workspace sizes are asked for without them).
struct Cut {
  bool prompt;     // by the prompts' kernel
  int block_shift; // log2 of a row block's query rows
  int rows;        // most of them in any
  int64_t blocks;  // at most this many row blocks (of each key-value head)
  int64_t chunks;  // at most this many chunks of any sequence's keys
  int64_t parts;   // at most this many partial results
};
Cut cut_call(const KvCache& c, const KvBatch& b, int ratio, int64_t prompt_min_rows) {
  Cut k;
  const int64_t rows = b.n_tokens * ratio;
  const int64_t each = prompt_min_rows < PROMPT_BLOCK ? prompt_min_rows : PROMPT_BLOCK;
  k.prompt = b.starts && rows * c.heads >= prompt_min_rows && rows >= each * b.batch;
  k.block_shift = k.prompt ? 7 : 4;
  static_assert(PROMPT_BLOCK == 1 << 7 && ATT_ROWS == 1 << 4, "rows of a row block");
  k.rows = b.starts || ratio > 1 << k.block_shift ? 1 << k.block_shift : ratio;
  k.blocks = b.starts ? row_blocks(b.n_tokens, ratio, k.block_shift) + b.batch : b.batch * row_blocks(1, ratio, k.block_shift);
  // Splitting costs a join (3 us in a table of up to 512 keys, against 2.6 us
  // for the keys) and a plan over the whole batch in every workgroup. With 1024
  // row blocks the GPU is full without it; then only a long table pays for the
  // balance that it brings to ragged lengths (us, split and not, 4 bits):
  // 1024 row blocks 2000 keys 41 / 35, 12000 keys 130 / 184; 2048 row blocks
  // 8000 keys 187 / 193, 12000 keys 329 / 286, 20000 keys 335 / 379; 8192 row
  // blocks 2000 keys 296 / 180.
  const int64_t keys = b.max_pages << c.shift, full = k.blocks * c.heads;
  const bool whole = keys <= ATT_UNSPLIT || (full >= 1024 && keys < 8 * full);
  k.chunks = whole ? 1 : (keys + ATT_MIN_CHUNK - 1) / ATT_MIN_CHUNK;
  const int64_t parts = 2 * (k.prompt ? PROMPT_TARGET : ATT_MAX_TARGET) / c.heads + 2;
  k.parts = k.chunks <= 1 ? 0 : parts / k.chunks < k.blocks ? parts : k.blocks * k.chunks;
  return k;
}
// At most this many units (see Seq).
int64_t call_units(const Cut& k, int heads, int target) {
  const int64_t spread = target / heads + 2 + k.blocks;
  return spread / k.chunks < k.blocks ? spread : k.blocks * k.chunks;
}

template <int BITS, int DP, bool FULL, bool SPLIT>
int launch_attend(const AttArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((kv_attend<BITS, DP, FULL, SPLIT>), dim3(unsigned(a.units * a.c.heads)), dim3(64 * ATT_WAVES), 0, s,
                     a);
  return launch_status();
}
template <int BITS, int DP>
int launch_attend(const AttArgs& a, bool split, hipStream_t s) {
  if (a.c.dim == DP)
    return split ? launch_attend<BITS, DP, true, true>(a, s) : launch_attend<BITS, DP, true, false>(a, s);
  return split ? launch_attend<BITS, DP, false, true>(a, s) : launch_attend<BITS, DP, false, false>(a, s);
}
template <int BITS>
int launch_attend(const AttArgs& a, bool split, hipStream_t s) {
  if (a.c.dim <= 64) return launch_attend<BITS, 64>(a, split, s);
  if (a.c.dim <= 128) return launch_attend<BITS, 128>(a, split, s);
  return launch_attend<BITS, 256>(a, split, s);
}

size_t attention_workspace(const gptq_kv_cache* cache, const gptq_kv_batch* batch, int64_t q_heads,
                           int64_t prompt_min_rows) {
  KvCache c;
  KvBatch b;
  if (kv_views(cache, batch, &c, &b) != GPTQ_OK || q_heads < 1 || q_heads > 65535 || q_heads % c.heads != 0) return 0;
  if (b.batch == 0 || b.n_tokens == 0) return 0;
  const Cut k = cut_call(c, b, int(q_heads / c.heads), prompt_min_rows);
  return size_t(k.parts) * size_t(c.heads) * size_t(k.rows) * (size_t(c.dim) * sizeof(float) + sizeof(float2));
}

// gptq_kv_attention with the rows from which on the prompts' kernel runs.
int attention(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const void* q, int q_dtype, int64_t q_heads,
              int64_t ldq, double scale, const float* slopes, void* out, int out_dtype, int64_t ldo, void* ws,
              size_t ws_bytes, int32_t* info, void* stream, int64_t prompt_min_rows) {
  AttArgs a{};
  int st = kv_views(cache, batch, &a.c, &a.b);
  if (st != GPTQ_OK) return st;
  const size_t eq = kv_elem_bytes(q_dtype), eo = kv_elem_bytes(out_dtype);
  if (eq == 0 || eo == 0 || q_heads < 1 || q_heads > 65535 || q_heads % a.c.heads != 0) return GPTQ_E_INVALID_ARG;
  const int64_t row = q_heads * a.c.dim;
  if (ldq < row || ldo < row || ldq > (int64_t(1) << 40) || ldo > (int64_t(1) << 40)) return GPTQ_E_INVALID_ARG;
  if (!(scale >= -3.0e38 && scale <= 3.0e38)) return GPTQ_E_INVALID_ARG;
  if (a.b.n_tokens > 0 && (!q || !out)) return GPTQ_E_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(q) % eq != 0 || reinterpret_cast<uintptr_t>(out) % eo != 0 ||
      reinterpret_cast<uintptr_t>(slopes) % 4 != 0)
    return GPTQ_E_INVALID_ARG;
  if (a.b.n_tokens == 0 || a.b.batch == 0) return GPTQ_OK;
  a.ratio = int(q_heads / a.c.heads);
  const Cut k = cut_call(a.c, a.b, a.ratio, prompt_min_rows);
  const bool split = q_dtype == GPTQ_F32 || out_dtype == GPTQ_F32;
  // One round of resident workgroups is what the keys are split for; prompts
  // have that many row blocks, and split only where a sequence is far longer
  // than the others.
  const int dp = a.c.dim <= 64 ? 64 : a.c.dim <= 128 ? 128 : 256;
  a.target = k.prompt ? PROMPT_TARGET : 256 * att_waves_per_simd(cache->bits, dp, split);
  const int64_t units = call_units(k, a.c.heads, a.target);
  // A launch has fewer than 2^32 threads (256 a workgroup, 512 in the prompts' kernel).
  if (units * a.c.heads >= (int64_t(1) << (k.prompt ? 23 : 24))) return GPTQ_E_INVALID_ARG;
  a.block_shift = k.block_shift;
  a.by_heads = Divider::by(uint32_t(a.c.heads));
  a.by_ratio = Divider::by(uint32_t(a.ratio));
  a.per_token = int(row_blocks(1, a.ratio, k.block_shift));
  a.rows = k.rows;
  a.splits = k.parts > 0;
  a.units = int(units);
  a.parts = int(k.parts);
  a.q = q;
  a.out = out;
  a.slopes = slopes;
  a.info = info;
  a.ldq = ldq;
  a.ldo = ldo;
  a.scale = float(scale * 1.4426950408889634);
  a.q_dtype = q_dtype;
  a.out_dtype = out_dtype;
  a.q_vec = kv_vec16(q, ldq, q_dtype);
  a.out_vec = kv_vec16(out, ldo, out_dtype);
  if (a.splits) {
    if (ws_bytes < attention_workspace(cache, batch, q_heads, prompt_min_rows)) return GPTQ_E_WORKSPACE;
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 16 != 0) return GPTQ_E_INVALID_ARG;
    a.part_o = static_cast<float*>(ws);  // its rows stay 16-byte aligned: head_dim is a multiple of 16
    a.part_ml = reinterpret_cast<float2*>(a.part_o + k.parts * a.c.heads * a.rows * a.c.dim);
  }
  hipStream_t s = as_stream(stream);
  st = k.prompt           ? launch_prompt(a, cache->bits, split, s)
       : cache->bits == 4 ? launch_attend<4>(a, split, s)
                          : launch_attend<8>(a, split, s);
  if (st != GPTQ_OK || !a.splits) return st;
  // A row block with several units has more than the mean share of the work,
  // so there are fewer than `target` of them (over all heads). Each gets a
  // workgroup a row, or fewer where that would be very many.
  const int64_t several = a.target / a.c.heads + 2, most = (several < k.blocks ? several : k.blocks) * a.c.heads;
  const int rows = most * a.rows <= JOIN_GROUPS ? a.rows : int((JOIN_GROUPS + most - 1) / most);
  hipLaunchKernelGGL(kv_join, dim3(unsigned(most * rows)), dim3(64 * ATT_WAVES), 0, s, a, rows);
  return launch_status();
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" size_t gptq_kv_attention_workspace_size(const gptq_kv_cache* cache, const gptq_kv_batch* batch,
                                                   int64_t q_heads) {
  return attention_workspace(cache, batch, q_heads, PROMPT_MIN_ROWS);
}

extern "C" int gptq_kv_attention(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const void* q, int q_dtype,
                                 int64_t q_heads, int64_t ldq, double scale, const float* slopes, void* out,
                                 int out_dtype, int64_t ldo, void* ws, size_t ws_bytes, int32_t* info, void* stream) {
  return attention(cache, batch, q, q_dtype, q_heads, ldq, scale, slopes, out, out_dtype, ldo, ws, ws_bytes, info, stream,
                   PROMPT_MIN_ROWS);
}
