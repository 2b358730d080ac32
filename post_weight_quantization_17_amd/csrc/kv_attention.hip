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
// is bound by the cache's bytes and by their conversion.
//
// Operands. The codes enter the MFMAs as integers: a 4-bit code c, moved to
// bits 6..9 of an fp16 half and OR-ed under the exponent of 16, is 16 + c
// exactly; an 8-bit one under the exponent of 1024 is 1024 + c. Scales and
// zeros stay outside:
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
// tiles skip the rescaling. Queries are scaled to a largest element of 2^13
// to 2^14, exact for 16-bit types (bf16's exponents do not fit fp16); the
// power of two is put back in fp32. fp32 queries, and weights for fp32
// outputs, are split into two fp16 parts, each with its own MFMA.
//
// Split. A workgroup's 4 waves take 32-key tiles in turn and are joined
// through LDS; where the rows alone do not fill the GPU, a row block's keys
// are split over workgroups too, whose partial sums kv_join adds in a fixed
// order. Each partial result has its M; all reductions are fp32.
#include "kv_cache.h"

namespace gptq {
namespace {

constexpr int ATT_WAVES = 4;
constexpr int ATT_ROWS = 16;                     // query rows of a workgroup
constexpr int ATT_TILE = 32;                     // keys a wave takes at a time
constexpr int ATT_MIN_CHUNK = 256;               // fewest keys of a workgroup when a row's keys are split
constexpr int ATT_MAX_SPLITS = 128;
constexpr int ATT_TARGET_GROUPS = 1024;          // workgroups that fill 256 CUs
constexpr float ATT_W_TOP = 8.0f;                // log2 of the largest weight after a rescaling
constexpr float ATT_W_LIMIT = 32768.0f;          // a weight above this asks for the next one
constexpr float ATT_LOWEST = -3.402823466e38f;   // M before the first key
constexpr float LOG2E = 1.44269504088896340736f;

struct AttArgs {
  KvCache c;
  KvBatch b;
  const void* q;
  void* out;
  const float* slopes;
  float* part_o;   // [splits][n_tokens][q_heads][dim]
  float2* part_ml; // [splits][n_tokens][q_heads]
  int32_t* info;
  int64_t ldq, ldo;
  float scale;  // of the scores, in log2 units
  int ratio;    // query heads that share a key-value head
  int q_dtype, out_dtype, q_vec;
  int splits;
};

// The row blocks of a sequence with n new tokens.
__host__ __device__ __forceinline__ int64_t row_blocks(int64_t n, int ratio) {
  return (n * ratio + ATT_ROWS - 1) / ATT_ROWS;
}

// How the keys [0, kend) of a row block are split: chunk keys a workgroup,
// `active` workgroups. Chunks are whole multiples of the 4 waves' tiles.
struct Split {
  int64_t chunk;
  int active;
};
__device__ __forceinline__ Split split_keys(int64_t kend, int splits) {
  constexpr int64_t step = ATT_WAVES * ATT_TILE;
  int64_t chunk = (kend + splits - 1) / splits;
  chunk = (chunk + step - 1) / step * step;
  if (chunk < ATT_MIN_CHUNK) chunk = ATT_MIN_CHUNK;
  const int64_t n = (kend + chunk - 1) / chunk;
  return Split{chunk, int(n < 1 ? 1 : n)};
}

// A sequence's share of the new tokens.
struct Seq {
  int64_t b;   // sequence, -1: none
  int64_t t0;  // its first token
  int64_t n;   // its new tokens
  int64_t rb;  // row block within it
};

// The sequence and row block that workgroup number `at` works on. Uniform
// over the wave, all of whose lanes take part.
__device__ __forceinline__ Seq find_block(const KvBatch& q, int ratio, int64_t at, int lane) {
  if (!q.starts) {
    const int64_t per = row_blocks(1, ratio);
    return Seq{at / per, at / per, 1, at % per};
  }
  int64_t before = 0;  // row blocks of the sequences passed
  for (int64_t b0 = 0; b0 < q.batch; b0 += 64) {
    const int64_t b = b0 + lane;
    int64_t t0 = 0, n = 0;
    if (b < q.batch) {
      t0 = q.starts[b];
      n = int64_t(q.starts[b + 1]) - t0;
      if (n < 0 || t0 < 0 || t0 + n > q.n_tokens) n = 0;
    }
    const int64_t mine = row_blocks(n, ratio);
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int64_t up = __shfl_up(sum, o);
      if (lane >= o) sum += up;
    }
    const uint64_t past = __ballot(before + sum > at);
    if (past != 0) {
      const int src = __ffsll((unsigned long long)past) - 1;
      const int64_t first = before + __shfl(sum - mine, src);
      return Seq{b0 + src, __shfl(t0, src), __shfl(n, src), at - first};
    }
    before += __shfl(sum, 63);
  }
  return Seq{-1, 0, 0, 0};
}

// Keys that row block rb of a sequence of `len` cached tokens, n of them
// new, can see: those of its last row.
__device__ __forceinline__ int64_t keys_seen(int64_t len, int64_t n, int64_t i, int64_t cap) {
  const int64_t end = len - n + i + 1;
  return end < 0 ? 0 : end > cap ? cap : end;
}
__device__ __forceinline__ int64_t block_last_row(int64_t n, int ratio, int64_t rb) {
  const int64_t last = rb * ATT_ROWS + ATT_ROWS - 1, rows = n * ratio;
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
  static constexpr float off = BITS == 4 ? 16.0f : 1024.0f;
  static constexpr uint32_t magic = BITS == 4 ? 0x4C004C00u : 0x64006400u;
  static constexpr int at = BITS == 4 ? 6 : 0;
};

// 4-bit codes: code i (0..3) of each 16-bit half of w, as two halves 16 + c.
template <int I>
__device__ __forceinline__ uint32_t nibbles(uint32_t w) {
  constexpr int up = 6 - 4 * I;
  return ((up > 0 ? w << up : w >> -up) & 0x03C003C0u) | Half<4>::magic;
}

// The 8 codes of a lane's k-slots in one MFMA of the first product. 4 bits:
// one word, in the order 0 4 1 5 2 6 3 7; 8 bits: two words, in order.
template <int BITS>
struct KeyOrder {
  static constexpr int code(int i) { return BITS == 4 ? (i % 2) * 4 + i / 2 : i; }
};
template <int BITS>
__device__ __forceinline__ void key_codes(const uint32_t* w, uint32_t (&h)[4]) {
  if constexpr (BITS == 4) {
    h[0] = nibbles<0>(w[0]);
    h[1] = nibbles<1>(w[0]);
    h[2] = nibbles<2>(w[0]);
    h[3] = nibbles<3>(w[0]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      h[2 * i] = __builtin_amdgcn_perm(0x64646464u, w[i], 0x04010400u);
      h[2 * i + 1] = __builtin_amdgcn_perm(0x64646464u, w[i], 0x04030402u);
    }
  }
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
  uint32_t ok;  // bit t: subtile t lies on a page
};

template <int BITS, int DP, bool FULL, bool SPLIT>
__global__ void __launch_bounds__(64 * ATT_WAVES)
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
  const int kv = int(blockIdx.x % unsigned(c.heads));
  const Seq sq = find_block(a.b, a.ratio, int64_t(blockIdx.x / unsigned(c.heads)), lane);
  if (sq.b < 0 || sq.b >= a.b.batch) return;  // whole workgroup; uniform

  const int64_t cap = a.b.max_pages << c.shift;
  const int64_t len = a.b.lens[sq.b];
  const int64_t last_row = block_last_row(sq.n, a.ratio, sq.rb);
  const int nrows = int(last_row - sq.rb * ATT_ROWS) + 1;
  const int64_t kend = keys_seen(len, sq.n, last_row / a.ratio, cap);
  if (len > cap && threadIdx.x == 0) kv_flag(a.info);
  const Split sp = split_keys(kend, a.splits);
  if (int(blockIdx.y) >= sp.active) return;
  const int64_t k0 = int64_t(blockIdx.y) * sp.chunk;
  const int64_t k1 = kend < k0 + sp.chunk ? kend : k0 + sp.chunk;

  // This lane's query row, and the keys that every row of the block sees.
  const int64_t row = sq.rb * ATT_ROWS + n16;
  const bool live = n16 < nrows;
  const int64_t i = live ? row / a.ratio : 0;
  const int hq = kv * a.ratio + (live ? int(row % a.ratio) : 0);
  const int64_t lim = live ? keys_seen(len, sq.n, i, cap) : 0;
  const int64_t all_see = keys_seen(len, sq.n, sq.rb * ATT_ROWS / a.ratio, cap);
  const int64_t pos = len - sq.n + i;
  const float slope = a.slopes ? a.slopes[hq] * LOG2E : 0.0f;

  // Queries: block j of 8 elements of this lane, in the order of the codes.
  const auto blk = [&](int j) { return FULL ? g * NJ + j : 4 * j + g; };
  half8 qh[NJ], ql[NJ];
  float qsum = 0.0f, row_scale;
  {
    float f[NJ][8];
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[j][e] = 0.0f;
      const int d0 = 8 * blk(j);
      if (live && d0 < c.dim) {
        const int64_t at = (sq.t0 + i) * a.ldq + int64_t(hq) * c.dim + d0;
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
    row_scale = ldexpf(a.scale, ex - 13);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = ldexpf(f[j][KeyOrder<BITS>::code(e)], 13 - ex);
        qh[j][e] = _Float16(s);
        qsum += float(qh[j][e]);
        if constexpr (SPLIT) ql[j][e] = _Float16(s - float(qh[j][e]));
      }
    qsum += __shfl_xor(qsum, 16);
    qsum += __shfl_xor(qsum, 32);
  }

  floatx4 o[DPL];
#pragma unroll
  for (int m = 0; m < DPL; ++m) o[m] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  float M = ATT_LOWEST, l = 0.0f;
  const int vc = n16 * DPL < c.dim ? n16 : 0;  // lanes past the head's end repeat the first one's codes

  const auto load = [&](int64_t p0, TL& t) {
    t.ok = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t p = p0 + 16 * u;
      int64_t id = -1;
      if (p < k1) id = kv_page(c, a.b, sq.b, p, a.info);
      if (id >= 0) t.ok |= 1u << u;
      // Keys on no page read the first page's rows, which are masked.
      const int64_t base = id < 0 ? int64_t(kv) << c.shift
                                  : ((id * c.heads + kv) << c.shift) + (p & ((int64_t(1) << c.shift) - 1));
      const uint32_t* kr = c.k_codes + base * c.words + n16 * c.words;
      if constexpr (FULL) {
#pragma unroll
        for (int w = 0; w < KW; ++w) t.k[u][w] = kr[g * KW + w];
      } else {
        constexpr int W = BITS / 4;  // words of a block
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int w = 0; w < W; ++w) t.k[u][W * j + w] = 8 * blk(j) < c.dim ? kr[W * blk(j) + w] : 0u;
      }
      t.kg[u] = *reinterpret_cast<const uint4*>(c.k_grid + base + 4 * g);
      t.vg[u] = *reinterpret_cast<const uint4*>(c.v_grid + base + 4 * g);
      if constexpr (SPLIT) t.kz[u] = c.k_grid[base + n16];
      const uint32_t* vr = c.v_codes + base * c.words + 4 * g * c.words;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (DPL * BITS == 16) {
          t.v[4 * u + r][0] = reinterpret_cast<const uint16_t*>(vr + r * c.words)[vc];
        } else {
#pragma unroll
          for (int w = 0; w < VW; ++w) t.v[4 * u + r][w] = vr[r * c.words + VW * vc + w];
        }
      }
    }
  };

  const auto compute = [&](int64_t p0, const TL& t) {
    float x[8], sv[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint32_t h[4];
        key_codes<BITS>(&t.k[u][j * (BITS / 4)], h);
        if constexpr (SPLIT) {
          const uint32_t z1 = MAGIC + (kv_zero<BITS>(t.kz[u]) * 0x10001u << Half<BITS>::at);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = as_u32(as_half2(h[e]) - as_half2(z1));
        }
        const half8 kc = as_half8(h[0], h[1], h[2], h[3]);
        if constexpr (SPLIT) acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(kc, ql[j], acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(kc, qh[j], acc, 0, 0, 0);
      }
      const uint32_t kg[4] = {t.kg[u].x, t.kg[u].y, t.kg[u].z, t.kg[u].w};
      const uint32_t vg[4] = {t.vg[u].x, t.vg[u].y, t.vg[u].z, t.vg[u].w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float s = kv_scale(kg[r]) * row_scale;
        x[4 * u + r] = SPLIT ? acc[r] * s : fmaf(-(OFF + float(kv_zero<BITS>(kg[r]))), qsum, acc[r]) * s;
        sv[4 * u + r] = kv_scale(vg[r]);
      }
    }
    if (a.slopes) {
      const float rel = float(int(p0 + 4 * g - pos));
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(slope, rel + float(16 * (e / 4) + e % 4), x[e]);
    }
    if (p0 + ATT_TILE > all_see || t.ok != 3u) {
      const int64_t left = lim - p0 - 4 * g;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool seen = 16 * (e / 4) + e % 4 < left && (t.ok >> (e / 4) & 1u) != 0;
        x[e] = seen ? x[e] : -INFINITY;
        sv[e] = seen ? sv[e] : 0.0f;
      }
    }
    float p[8], w[8], big = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p[e] = __builtin_amdgcn_exp2f(x[e] - M);
      w[e] = p[e] * sv[e];
      big = fmaxf(big, w[e]);
    }
    if (__any(big > ATT_W_LIMIT)) {
      float top = ATT_LOWEST;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, x[e] + __builtin_amdgcn_logf(sv[e]) - ATT_W_TOP);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      top = fmaxf(top, M);
      const float f = __builtin_amdgcn_exp2f(M - top);
      M = top;
      l *= f;
#pragma unroll
      for (int m = 0; m < DPL; ++m) o[m] *= f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = __builtin_amdgcn_exp2f(x[e] - M);
        w[e] = p[e] * sv[e];
      }
    }
    half8 wh, wl;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      l += p[e];
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
        for (int e = 0; e < 4; ++e) h[e] = nibbles<0>(lo[e]);
        product(8 * vw + 0, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = nibbles<1>(lo[e]);
        product(8 * vw + 1, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = nibbles<2>(lo[e]);
        product(8 * vw + 2, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = nibbles<3>(lo[e]);
        product(8 * vw + 3, h);
        if constexpr (DPL > 4) {
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = nibbles<0>(hi[e]);
          product(8 * vw + 4, h);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = nibbles<1>(hi[e]);
          product(8 * vw + 5, h);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = nibbles<2>(hi[e]);
          product(8 * vw + 6, h);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = nibbles<3>(hi[e]);
          product(8 * vw + 7, h);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = __builtin_amdgcn_perm(0x64646464u, lo[e], 0x04020400u);
        product(4 * vw + 0, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = __builtin_amdgcn_perm(0x64646464u, lo[e], 0x04030401u);
        product(4 * vw + 1, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = __builtin_amdgcn_perm(0x64646464u, hi[e], 0x04020400u);
        product(4 * vw + 2, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = __builtin_amdgcn_perm(0x64646464u, hi[e], 0x04030401u);
        product(4 * vw + 3, h);
      }
    }
  };

  // The next tile's loads are in flight while a tile is computed.
  const int64_t step = ATT_WAVES * ATT_TILE;
  int64_t p0 = k0 + wave * ATT_TILE;
  if (p0 < k1) {
    TL cur;
    load(p0, cur);
    for (; p0 < k1; p0 += step) {
      TL next;
      if (p0 + step < k1) load(p0 + step, next);
      compute(p0, cur);
      cur = next;
    }
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
    const int64_t at = sq.rb * ATT_ROWS + r;
    const int64_t t = sq.t0 + at / a.ratio;
    const int h = kv * a.ratio + int(at % a.ratio);
    float top = lds_m[0][r];
    for (int w = 1; w < ATT_WAVES; ++w) top = fmaxf(top, lds_m[w][r]);
    float sum = 0.0f;
    for (int w = 0; w < ATT_WAVES; ++w) sum += lds_l[w][r] * __builtin_amdgcn_exp2f(lds_m[w][r] - top);
    const int64_t heads_q = int64_t(c.heads) * a.ratio;
    if (sp.active > 1) {
      const int64_t pr = (int64_t(blockIdx.y) * a.b.n_tokens + t) * heads_q + h;
      for (int d = lane; d < c.dim; d += 64)
        a.part_o[pr * c.dim + d] = lds_o[0][r][d] + lds_o[1][r][d];
      if (lane == 0) a.part_ml[pr] = float2{top, sum};
    } else {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a row that sees no key gives zeros
      for (int d = lane; d < c.dim; d += 64) {
        const float v = (lds_o[0][r][d] + lds_o[1][r][d]) * inv;
        const int64_t oo = t * a.ldo + int64_t(h) * c.dim + d;
        if (a.out_dtype == GPTQ_F16)
          static_cast<_Float16*>(a.out)[oo] = from_f32<_Float16>(v);
        else if (a.out_dtype == GPTQ_BF16)
          static_cast<bf16*>(a.out)[oo] = from_f32<bf16>(v);
        else
          static_cast<float*>(a.out)[oo] = v;
      }
    }
  }
}

// Joins the splits of one row (token, query head), in their order: each wave
// adds every fourth one, and the waves' sums are added in order.
__global__ void __launch_bounds__(64 * ATT_WAVES)
kv_join(AttArgs a) {
  __shared__ float sums[ATT_WAVES][256];
  const KvCache& c = a.c;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t heads_q = int64_t(c.heads) * a.ratio;
  const int64_t t = int64_t(blockIdx.x) / heads_q;
  const int h = int(int64_t(blockIdx.x) % heads_q);
  // The token's sequence, and the keys of its row block as kv_attend took them.
  int64_t b = t, t0 = t, n = 1;
  if (a.b.starts) {
    int64_t cnt = 0;
    for (int64_t i0 = 0; i0 <= a.b.batch; i0 += 64) {
      const int64_t i = i0 + lane;
      const uint64_t le = __ballot(i <= a.b.batch && int64_t(a.b.starts[i <= a.b.batch ? i : 0]) <= t);
      cnt += __popcll(le);
      if (le != ~uint64_t(0)) break;
    }
    b = cnt - 1;
    if (b < 0 || b >= a.b.batch) return;
    t0 = a.b.starts[b];
    n = int64_t(a.b.starts[b + 1]) - t0;
    if (n < 0 || t0 < 0 || t0 + n > a.b.n_tokens || t < t0 || t >= t0 + n) return;
  }
  const int64_t cap = a.b.max_pages << c.shift;
  const int64_t rb = ((t - t0) * a.ratio + h % a.ratio) / ATT_ROWS;
  const int64_t kend = keys_seen(a.b.lens[b], n, block_last_row(n, a.ratio, rb) / a.ratio, cap);
  const Split sp = split_keys(kend, a.splits);
  if (sp.active <= 1) return;  // kv_attend wrote the row

  const int64_t stride = a.b.n_tokens * heads_q, pr = t * heads_q + h;
  float top = ATT_LOWEST;
  for (int s = 0; s < sp.active; ++s) top = fmaxf(top, a.part_ml[s * stride + pr].x);
  float sum = 0.0f, o[4] = {};
  for (int s = 0; s < sp.active; ++s) {
    const float2 ml = a.part_ml[s * stride + pr];
    const float f = __builtin_amdgcn_exp2f(ml.x - top);
    sum += ml.y * f;
    if (s % ATT_WAVES == wave) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = lane + 64 * e;
        if (d < c.dim) o[e] = fmaf(a.part_o[(s * stride + pr) * c.dim + d], f, o[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sums[wave][lane + 64 * e] = o[e];
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= c.dim) return;
  float v = sums[0][d];
  for (int w = 1; w < ATT_WAVES; ++w) v += sums[w][d];
  v *= sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t oo = t * a.ldo + int64_t(h) * c.dim + d;
  if (a.out_dtype == GPTQ_F16)
    static_cast<_Float16*>(a.out)[oo] = from_f32<_Float16>(v);
  else if (a.out_dtype == GPTQ_BF16)
    static_cast<bf16*>(a.out)[oo] = from_f32<bf16>(v);
  else
    static_cast<float*>(a.out)[oo] = v;
}

// Row blocks of a call (at most this many) times key-value heads.
int64_t call_blocks(const KvCache& c, const KvBatch& b, int ratio) {
  const int64_t rows = b.starts ? row_blocks(b.n_tokens, ratio) + b.batch : b.batch * row_blocks(1, ratio);
  return rows * c.heads;
}

// Workgroups a row block's keys may be split over: enough of them to fill
// the GPU, none with less than ATT_MIN_CHUNK of the table's keys.
int call_splits(const KvCache& c, const KvBatch& b, int ratio) {
  const int64_t blocks = call_blocks(c, b, ratio);
  if (blocks < 1) return 1;
  const int64_t keys = b.max_pages << c.shift;
  int64_t s = (ATT_TARGET_GROUPS + blocks - 1) / blocks;
  const int64_t most = (keys + ATT_MIN_CHUNK - 1) / ATT_MIN_CHUNK;
  if (s > most) s = most;
  if (s > ATT_MAX_SPLITS) s = ATT_MAX_SPLITS;
  return int(s < 1 ? 1 : s);
}

template <int BITS, int DP, bool FULL, bool SPLIT>
int launch_attend(const AttArgs& a, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL((kv_attend<BITS, DP, FULL, SPLIT>), grid, dim3(64 * ATT_WAVES), 0, s, a);
  return launch_status();
}
template <int BITS, int DP>
int launch_attend(const AttArgs& a, dim3 grid, bool split, hipStream_t s) {
  if (a.c.dim == DP)
    return split ? launch_attend<BITS, DP, true, true>(a, grid, s)
                 : launch_attend<BITS, DP, true, false>(a, grid, s);
  return split ? launch_attend<BITS, DP, false, true>(a, grid, s)
               : launch_attend<BITS, DP, false, false>(a, grid, s);
}
template <int BITS>
int launch_attend(const AttArgs& a, dim3 grid, bool split, hipStream_t s) {
  if (a.c.dim <= 64) return launch_attend<BITS, 64>(a, grid, split, s);
  if (a.c.dim <= 128) return launch_attend<BITS, 128>(a, grid, split, s);
  return launch_attend<BITS, 256>(a, grid, split, s);
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" size_t gptq_kv_attention_workspace_size(const gptq_kv_cache* cache, const gptq_kv_batch* batch,
                                                   int64_t q_heads) {
  KvCache c;
  KvBatch b;
  if (kv_views(cache, batch, &c, &b) != GPTQ_OK || q_heads < 1 || q_heads % c.heads != 0) return 0;
  const int splits = call_splits(c, b, int(q_heads / c.heads));
  if (splits <= 1) return 0;
  return size_t(splits) * size_t(b.n_tokens) * size_t(q_heads) * (size_t(c.dim) * sizeof(float) + sizeof(float2));
}

extern "C" int gptq_kv_attention(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const void* q, int q_dtype,
                                 int64_t q_heads, int64_t ldq, double scale, const float* slopes, void* out,
                                 int out_dtype, int64_t ldo, void* ws, size_t ws_bytes, int32_t* info, void* stream) {
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
  const int64_t blocks = call_blocks(a.c, a.b, a.ratio);
  if (blocks >= (int64_t(1) << 24) || a.b.n_tokens * q_heads >= (int64_t(1) << 31)) return GPTQ_E_INVALID_ARG;
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
  a.splits = call_splits(a.c, a.b, a.ratio);
  if (a.splits > 1) {
    if (ws_bytes < gptq_kv_attention_workspace_size(cache, batch, q_heads)) return GPTQ_E_WORKSPACE;
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 16 != 0) return GPTQ_E_INVALID_ARG;
    a.part_ml = static_cast<float2*>(ws);
    a.part_o = reinterpret_cast<float*>(a.part_ml + int64_t(a.splits) * a.b.n_tokens * q_heads);
  }
  const bool split = q_dtype == GPTQ_F32 || out_dtype == GPTQ_F32;
  const dim3 grid(unsigned(blocks), unsigned(a.splits));
  hipStream_t s = as_stream(stream);
  st = cache->bits == 4 ? launch_attend<4>(a, grid, split, s) : launch_attend<8>(a, grid, split, s);
  if (st != GPTQ_OK || a.splits == 1) return st;
  hipLaunchKernelGGL(kv_join, dim3(unsigned(a.b.n_tokens * q_heads)), dim3(64 * ATT_WAVES), 0, s, a);
  return launch_status();
}
