// What the attention kernels share: the work's division, and the pieces of
// the matrix products.
//
// Rows. The G query heads of a key head and a request's n nodes are n * G
// rows that read the same keys; row = node * G + head. A tile is RT of them.
//
// Division of the work. A unit is one tile times one block of KB keys; the
// units of a call stand in one line (request, key head, tile, block), and
// each of B workgroups takes an equal stretch of it, whatever the requests'
// lengths. A tile whose blocks fall to several workgroups leaves partial
// results (sum of weighted values, maximum, sum), at most two per workgroup:
// slot 0 for a tile that began before its stretch, slot 1 for one that goes
// on after it. A second launch joins them in the line's order. The lengths
// are on the device, so every workgroup works the line out for itself: one
// prefix sum over the requests.
#pragma once

#include <math.h>

#include "k3_kv.h"

namespace k3 {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The running maximum is raised only by more than this (in powers of two):
// weights up to 2^8 are exact as ever in fp32 and bf16, and the output is
// rescaled a handful of times instead of at every block.
constexpr float kSlack = 8.f;
// fp16 weights are kept 2^6 higher, so that small ones stay normal numbers;
// with the slack they reach 2^14, under fp16's 65504.
template <bool BF>
constexpr float kLift = BF ? 0.f : 6.f;

// ---- the line of units ----------------------------------------------------

struct Request {
  int t0, n, len;  // first token, nodes, places
};
__device__ __forceinline__ Request request_of(const AttnArgs &a, int r) {
  Request q;
  q.t0 = a.cu[r];
  q.n = a.cu[r + 1] - q.t0;
  if (q.t0 < 0 || q.n < 0 || (long long)q.t0 + q.n > a.T) q.n = 0;
  q.len = a.kv_lens[r];
  if (q.len < 0 || q.len > a.blocks * a.c.page_size) q.len = 0;
  return q;
}
template <int RT>
__device__ __forceinline__ int tiles_of(const AttnArgs &a, int n) {
  return (int)(((long long)n * a.G + RT - 1) / RT);
}
template <int KB>
__device__ __forceinline__ int blocks_of(int len) {
  return len > 0 ? (len - 1) / KB + 1 : 1;
}
template <int RT, int KB>
__device__ __forceinline__ long long units_of(const AttnArgs &a, int r) {
  const Request q = request_of(a, r);
  return (long long)tiles_of<RT>(a, q.n) * a.c.n_heads * blocks_of<KB>(q.len);
}

// pre[r] = units before request r, pre[R] = all of them; a workgroup of
// THREADS threads. Ends with a barrier.
template <int RT, int KB, int THREADS>
__device__ __forceinline__ void line_of_units(const AttnArgs &a, long long *pre) {
  const int tid = threadIdx.x, lane = tid & 63;
  __shared__ long long wave_sum[THREADS / 64];
  if (a.R == 1) {
    if (tid == 0) {
      pre[0] = 0;
      pre[1] = units_of<RT, KB>(a, 0);
    }
    __syncthreads();
    return;
  }
  const int per = (a.R + THREADS - 1) / THREADS;
  const int lo = min(a.R, tid * per), hi = min(a.R, lo + per);
  long long own = 0;
  for (int r = lo; r < hi; r++) {
    pre[r] = own;
    own += units_of<RT, KB>(a, r);
  }
  long long incl = own;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const long long x = __shfl_up(incl, m);
    if (lane >= m) incl += x;
  }
  if (lane == 63) wave_sum[tid >> 6] = incl;
  __syncthreads();
  long long base = incl - own;
  for (int w = 0; w < (tid >> 6); w++) base += wave_sum[w];
  for (int r = lo; r < hi; r++) pre[r] += base;
  if (hi == a.R && lo < hi) pre[a.R] = base + own;
  __syncthreads();
}

// The request that unit u belongs to: the last r with pre[r] <= u.
__device__ __forceinline__ int request_at(const long long *pre, int R, long long u) {
  int lo = 0, hi = R - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A tile in the line.
struct Tile {
  Request q;
  int r, h, row0, blocks;
  long long first;  // its first unit
};
template <int RT, int KB>
__device__ __forceinline__ Tile tile_at(const AttnArgs &a, const long long *pre, long long u) {
  Tile t;
  t.r = request_at(pre, a.R, u);
  t.q = request_of(a, t.r);
  t.blocks = blocks_of<KB>(t.q.len);
  const long long x = u - pre[t.r];
  const long long tile = x / t.blocks;
  t.first = pre[t.r] + tile * t.blocks;
  const int tiles = tiles_of<RT>(a, t.q.n);
  t.h = (int)(tile / tiles);
  t.row0 = (int)(tile - (long long)t.h * tiles) * RT;
  return t;
}

__device__ __forceinline__ long long stretch(long long units, int b, int B) { return units * b / B; }

// ---- partial results --------------------------------------------------------

// part: for 2 B slots [RT][D] sums, then for each slot [RT] maxima, [RT] sums.
template <int RT, int D>
__device__ __forceinline__ float *part_o(const AttnArgs &a, int slot, int row) {
  return a.part + ((size_t)slot * RT + row) * D;
}
template <int RT, int D>
__device__ __forceinline__ float *part_ml(const AttnArgs &a, int B, int slot) {
  return a.part + (size_t)2 * B * RT * D + (size_t)slot * 2 * RT;
}
inline size_t part_bytes(int RT, int D, int B) { return (size_t)2 * B * RT * (D + 2) * sizeof(float); }

// ---- numbers ----------------------------------------------------------------

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const f32x2 v = {x, y};
  if (BF) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}
// Two e4m3 values (exact in either 16-bit type): bytes 0, 1 or 2, 3 of w.
template <bool BF, bool HI>
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
  if (BF) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, HI));
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, HI));
}
template <bool BF>
__device__ __forceinline__ f32x4 mfma16(u32x4 x, u32x4 y, f32x4 c) {
  if (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0,
                                                   0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0,
                                                0);
}
// Bits of the halves of w that are not finite numbers, as a mask of halves.
template <bool BF>
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
  constexpr uint32_t E = BF ? 0x7f80u : 0x7c00u;
  uint32_t m = 0;
  if ((w & E) == E) m |= 0xffffu;
  if ((w & (E << 16)) == (E << 16)) m |= 0xffff0000u;
  return m;
}
template <bool BF>
__device__ __forceinline__ float half_at(uint32_t w, int hi) {
  if (BF) return __builtin_bit_cast(float, hi ? w & 0xffff0000u : w << 16);
  return (float)__builtin_bit_cast(f16x2, w)[hi];
}
// Orders a wave's own LDS accesses, which its lanes share (LDS serves a
// wave's accesses in order; this keeps the compiler to that order).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// x of this lane and of lane l ^ 32 (l ^ 16), in either order: the swap of
// halves (of rows) of two copies leaves one in each.
struct Pair {
  float a, b;
};
__device__ __forceinline__ Pair with_xor32(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const u32x2 s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t a = s[0], b = s[1];  // (a bit cast of s[1] itself would take s[0])
  return {__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ __forceinline__ Pair with_xor16(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const u32x2 s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t a = s[0], b = s[1];
  return {__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ __forceinline__ float max_xor32(float x) {
  const Pair p = with_xor32(x);
  return fmaxf(p.a, p.b);
}
__device__ __forceinline__ float max_xor16(float x) {
  const Pair p = with_xor16(x);
  return fmaxf(p.a, p.b);
}
__device__ __forceinline__ float sum_xor32(float x) {
  const Pair p = with_xor32(x);
  return p.a + p.b;
}
__device__ __forceinline__ float sum_xor16(float x) {
  const Pair p = with_xor16(x);
  return p.a + p.b;
}

// Which of the 32 places from k0 on node i sees (present: those in a page).
__device__ __forceinline__ uint32_t word_of(const AttnArgs &a, const Request &q, int i, int w) {
  if (w < 0) return 0xffffffffu;
  if (a.mask) return w < a.words ? (uint32_t)a.mask[(size_t)(q.t0 + i) * a.words + w] : 0u;
  const int k = i + 1 - 32 * w;
  return k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1;
}
__device__ __forceinline__ uint32_t seen(const AttnArgs &a, const Request &q, int i, int k0, uint32_t present) {
  const int node = k0 - (q.len - q.n);
  const int w = node >> 5, sh = node & 31;
  const uint32_t lo = word_of(a, q, i, w);
  if (!sh) return lo & present;
  return ((lo >> sh) | (word_of(a, q, i, w + 1) << (32 - sh))) & present;
}

}  // namespace k3
