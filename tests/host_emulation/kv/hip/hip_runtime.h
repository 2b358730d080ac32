// Host emulation of the part of the HIP execution model that the key-value
// cache kernels use, for bounds-checked CPU runs of the library's own kernel
// source under AddressSanitizer (test infrastructure, never part of the
// library).
//
// Every workgroup runs as blockDim.x host threads; workgroups run one after
// another, so `__shared__` arrays become function-local statics. Cross-lane
// operations exchange values through a per-wave buffer behind a 64-thread
// barrier, so every lane of a wave must reach them together, as on the
// hardware. Global memory is the caller's host memory: an access outside an
// allocation is an ASan report.
#pragma once

#include <barrier>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <memory>
#include <thread>
#include <type_traits>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static
#define KV_OPAQUE_S(x) ((void)(x))
#define KV_OPAQUE_V(x) ((void)(x))
#define KV_FRESH_V(x) ((void)(x))

struct dim3 {
  uint32_t x, y, z;
  constexpr dim3(uint32_t x_ = 1, uint32_t y_ = 1, uint32_t z_ = 1) : x(x_), y(y_), z(z_) {}
};
struct alignas(16) uint4 {
  uint32_t x, y, z, w;
};
struct alignas(8) uint2 {
  uint32_t x, y;
};
struct alignas(8) float2 {
  float x, y;
};
struct alignas(16) float4 {
  float x, y, z, w;
};

typedef enum hipError_t { hipSuccess = 0 } hipError_t;
typedef struct ihipStream_t* hipStream_t;
inline hipError_t hipGetLastError() { return hipSuccess; }

namespace simt {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float floatx4_t __attribute__((ext_vector_type(4)));

struct Wave {
  std::barrier<> bar{64};
  int64_t v[2][64];
  half8_t a[2][64], b[2][64];
};
struct Workgroup {
  explicit Workgroup(unsigned n) : bar(n), waves((n + 63) / 64) {
    for (auto& w : waves) w = std::make_unique<Wave>();
  }
  std::barrier<> bar;
  std::vector<std::unique_ptr<Wave>> waves;
};

inline thread_local dim3 tid, bid;
inline thread_local Workgroup* wg = nullptr;
inline thread_local unsigned phase = 0;
inline dim3 grid_dim, block_dim;

inline Wave& my_wave() { return *wg->waves[tid.x / 64]; }
inline int my_lane() { return int(tid.x % 64); }

// Publishes v and returns the buffer that holds every lane's value. Double
// buffered: it is written again only after every lane has passed the next
// exchange's barrier.
inline const int64_t* exchange(int64_t v) {
  Wave& w = my_wave();
  const int p = int(phase++ & 1);
  w.v[p][my_lane()] = v;
  w.bar.arrive_and_wait();
  return w.v[p];
}
template <typename T>
inline T from_lane(T v, int src) {
  int64_t bits = 0;
  std::memcpy(&bits, &v, sizeof(T));
  const int64_t got = exchange(bits)[src];
  T r;
  std::memcpy(&r, &got, sizeof(T));
  return r;
}
inline int dpp_source(int lane, int ctrl) {
  const int row = lane & ~15, r = lane & 15;
  if (ctrl >= 0 && ctrl <= 0xFF) return (lane & ~3) | ((ctrl >> (2 * (lane & 3))) & 3);
  if (ctrl == 0x140) return row + (15 - r);
  if (ctrl == 0x141) return row + ((r & 8) | (7 - (r & 7)));
  if (ctrl >= 0x150 && ctrl <= 0x15F) return row + (ctrl - 0x150);
  std::fprintf(stderr, "host emulation: DPP control 0x%x not modelled\n", ctrl);
  std::abort();
}

// A DPP move that keeps `old` where the source lane is outside its row, where
// a row has nothing broadcast to it, or where the row mask excludes it.
inline int update_dpp(int old, int src, int ctrl, int row_mask, int bank_mask) {
  const int64_t* v = exchange(src);
  const int l = my_lane(), row = l / 16, r = l % 16;
  if (bank_mask != 0xf) std::abort();
  if (!(row_mask >> row & 1)) return old;
  if (ctrl >= 0x111 && ctrl <= 0x11F) return r >= ctrl - 0x110 ? int(v[l - (ctrl - 0x110)]) : old;  // row_shr
  if (ctrl == 0x142) return row > 0 ? int(v[16 * row - 1]) : old;                                   // row_bcast:15
  if (ctrl == 0x143) return l >= 32 ? int(v[31]) : old;                                             // row_bcast:31
  return int(v[dpp_source(l, ctrl)]);
}

// v_mfma_f32_16x16x32_f16: lane l holds A[l % 16][8 (l / 16) + j] and
// B[8 (l / 16) + j][l % 16], j = 0..7; it returns D[4 (l / 16) + r][l % 16].
inline floatx4_t mfma_16x16x32(half8_t a, half8_t b, floatx4_t c) {
  Wave& w = my_wave();
  const int l = my_lane(), p = int(phase++ & 1);
  w.a[p][l] = a;
  w.b[p][l] = b;
  w.bar.arrive_and_wait();
  const int n = l & 15, i0 = 4 * (l >> 4);
  floatx4_t d;
  for (int r = 0; r < 4; ++r) {
    float acc = c[r];
    for (int k = 0; k < 32; ++k)
      acc = std::fmaf(float(w.a[p][16 * (k / 8) + i0 + r][k % 8]), float(w.b[p][16 * (k / 8) + n][k % 8]), acc);
    d[r] = acc;
  }
  return d;
}

inline uint32_t perm(uint32_t s0, uint32_t s1, uint32_t sel) {
  const uint64_t bytes = uint64_t(s0) << 32 | s1;
  uint32_t r = 0;
  for (int i = 0; i < 4; ++i) {
    const uint32_t k = (sel >> (8 * i)) & 0xFF;
    if (k > 7) {
      std::fprintf(stderr, "host emulation: byte selector %u not modelled\n", k);
      std::abort();
    }
    r |= uint32_t((bytes >> (8 * k)) & 0xFF) << (8 * i);
  }
  return r;
}

template <typename K, typename... A>
void launch(K kernel, dim3 grid, dim3 block, A... args) {
  if (grid.z != 1 || block.y != 1 || block.z != 1 || block.x % 64 != 0 || block.x > 1024) {
    std::fprintf(stderr, "host emulation: launch shape not modelled\n");
    std::abort();
  }
  grid_dim = grid;
  block_dim = block;
  for (uint32_t by = 0; by < grid.y; ++by)
    for (uint32_t bx = 0; bx < grid.x; ++bx) {
      Workgroup g(block.x);
      std::vector<std::thread> th;
      th.reserve(block.x);
      for (uint32_t t = 0; t < block.x; ++t)
        th.emplace_back([&, t] {
          tid = dim3(t);
          bid = dim3(bx, by);
          wg = &g;
          phase = 0;
          kernel(args...);
        });
      for (auto& x : th) x.join();
    }
}

}  // namespace simt

#define threadIdx (simt::tid)
#define blockIdx (simt::bid)
#define gridDim (simt::grid_dim)
#define blockDim (simt::block_dim)

inline void __syncthreads() { simt::wg->bar.arrive_and_wait(); }

inline float __int_as_float(int v) {
  float f;
  std::memcpy(&f, &v, 4);
  return f;
}
inline int __float_as_int(float f) {
  int v;
  std::memcpy(&v, &f, 4);
  return v;
}
inline float __uint_as_float(uint32_t v) { return __int_as_float(int(v)); }
inline uint32_t __float_as_uint(float f) { return uint32_t(__float_as_int(f)); }
inline int __popcll(uint64_t v) { return __builtin_popcountll(v); }
inline int __ffsll(unsigned long long v) { return __builtin_ffsll((long long)v); }

inline uint64_t __ballot(bool p) {
  const int64_t* v = simt::exchange(p);
  uint64_t m = 0;
  for (int i = 0; i < 64; ++i) m |= uint64_t(v[i] != 0) << i;
  return m;
}
inline bool __any(bool p) { return __ballot(p) != 0; }
template <typename T>
inline T __shfl_xor(T v, int mask) {
  return simt::from_lane(v, simt::my_lane() ^ mask);
}
template <typename T>
inline T __shfl_up(T v, int by) {
  const int l = simt::my_lane();
  return simt::from_lane(v, l < by ? l : l - by);
}
template <typename T>
inline T __shfl(T v, int src) {
  return simt::from_lane(v, src);
}

#define __builtin_amdgcn_update_dpp(old, src, ctrl, rm, bm, bc) simt::update_dpp((old), (src), (ctrl), (rm), (bm))
#define __builtin_amdgcn_mov_dpp(src, ctrl, rm, bm, bc) simt::from_lane((src), simt::dpp_source(simt::my_lane(), (ctrl)))
#define __builtin_amdgcn_readlane(v, src) simt::from_lane((v), (src))
#define __builtin_amdgcn_readfirstlane(v) simt::from_lane((v), 0)
#define __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, cbsz, abid, blgp) simt::mfma_16x16x32((a), (b), (c))
#define __builtin_amdgcn_perm(s0, s1, sel) simt::perm((s0), (s1), (sel))
#define __builtin_amdgcn_rcpf(x) (1.0f / (x))
#define __builtin_amdgcn_fmed3f(x, lo, hi) std::fmax(std::fmin((x), (hi)), (lo))
#define __builtin_amdgcn_exp2f(x) std::exp2f(x)
#define __builtin_amdgcn_logf(x) std::log2f(x)

#define hipLaunchKernelGGL(kernel, grid, block, shmem, stream, ...) \
  simt::launch((kernel), dim3(grid), dim3(block), __VA_ARGS__)
