// What the attention kernels share: the work's division, and the pieces of
// the matrix products.
//
// Rows. The G query heads of a key head and a request's n nodes are n * G
// rows that read the same keys; row = node * G + head. A tile is RT of them.
//
// Division of the work. The tiles of a call stand in one line (request, key
// head, tile), each as long as the places that its rows may see, and each of
// B workgroups takes an equal stretch of the line, in whole blocks of KB
// places, whatever the requests' lengths. A tile whose blocks fall to several
// workgroups leaves partial results (sum of weighted values, maximum, sum), at
// most two per workgroup: slot 0 for a tile that began before its stretch,
// slot 1 for one that goes on after it. A second launch joins them in the
// line's order. The lengths are on the device, so every workgroup works the
// line out for itself: one prefix sum over the requests, and a closed form
// within each.
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

// A block for a tile of up to half the waves' rows takes 11 / 16 of the time
// of a full one, and what a tile takes apart from its blocks is that of so
// many places: its tables, queries and first blocks come one after the other
// (14 us, at 1.8 us for 64 places of a head of 128).
constexpr int kHalfCost = 11;
template <int RT>
constexpr int kFixedPlaces = RT < 128 ? 128 : 512;
constexpr int kMaxWorkgroups = 1024;  // of a launch: at most two to a CU
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The running maximum is raised only by more than this (in powers of two):
// weights up to 2^8 are exact as ever in fp32 and bf16, and the output is
// rescaled a handful of times instead of at every block. (The sums of weighted
// values pass fp32's range 2^8 earlier: bf16 values beyond 2^119 may overflow
// there where their average would not.)
constexpr float kSlack = 8.f;
// fp16 weights are kept 2^6 higher, so that small ones stay normal numbers;
// with the slack they reach 2^14, under fp16's 65504.
template <bool BF>
constexpr float kLift = BF ? 0.f : 6.f;

// ---- the line ---------------------------------------------------------------

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

// Row `row`'s node (its head in the group: row - node * G).
__device__ __forceinline__ int node_of(const AttnArgs &a, int row) {
  return (int)(__umulhi(2u * (uint32_t)row, a.group_magic) >> a.group_shift);
}

// (No divisions in what follows: a workgroup's way to its first block is a few
// hundred instructions that it runs once, and each 64-bit division is a
// hundred more to fetch.)
// The cost of a request's tiles, in sixteenths of a place: what each has
// fixed, the first tile's places, what each next one has more. The last one's
// places count for less if it is of up to HALF rows. T * Hq <= 2^30 rows and
// 2^30 places keep all sums below 2^61.
template <int RT, int HALF>
struct Cost {
  int tiles, last_rows;
  long long base, slope, all;
  static constexpr long long kFixed = 16 * kFixedPlaces<RT>;
  __device__ __forceinline__ Cost(const AttnArgs &a, const Request &q) {
    const long long rows = (long long)q.n * a.G;
    tiles = (int)((rows + RT - 1) / RT);
    last_rows = (int)(rows - (long long)(tiles - 1) * RT);
    const bool causal = !a.mask && q.len >= q.n;
    slope = causal ? a.slope : 0;
    base = 16ll * (causal ? q.len - q.n : q.len) + slope;
    all = tiles ? of_first(tiles - 1) + of(tiles - 1) : 0;
  }
  // a place's cost; the first x tiles of a key head; tile x
  __device__ __forceinline__ int weight(int x) const { return x == tiles - 1 && last_rows <= HALF ? kHalfCost : 16; }
  __device__ __forceinline__ long long of_first(long long x) const {
    return x * (kFixed + base) + slope * (x * (x - 1) / 2);
  }
  __device__ __forceinline__ long long of(int x) const { return kFixed + ((base + slope * x) * weight(x) >> 4); }
  __device__ __forceinline__ long long of_request(const AttnArgs &a) const { return all * a.c.n_heads; }
};

// The requests go to the THREADS threads of a workgroup in runs of `per`.
// pre[i] = cost before thread i's, pre[THREADS] = all of it. Ends with a
// barrier.
template <int THREADS>
struct Line {
  long long pre[THREADS + 1], wave_sum[THREADS / 64];
  Request request[THREADS];  // the last of each thread's
};
template <int THREADS>
__device__ __forceinline__ int run_of(int R) { return (R + THREADS - 1) / THREADS; }

template <int RT, int HALF, int THREADS>
__device__ __forceinline__ void line_of_tiles(const AttnArgs &a, Line<THREADS> &L) {
  const int tid = threadIdx.x, lane = tid & 63, per = run_of<THREADS>(a.R);
  long long own = 0;
  for (int r = tid * per; r < min(a.R, tid * per + per); r++) {
    const Request q = request_of(a, r);
    own += Cost<RT, HALF>(a, q).of_request(a);
    L.request[tid] = q;
  }
  long long incl = own;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const long long x = __shfl_up(incl, m);
    if (lane >= m) incl += x;
  }
  if (lane == 63) L.wave_sum[tid >> 6] = incl;
  __syncthreads();
  long long base = incl - own;
  for (int w = 0; w < (tid >> 6); w++) base += L.wave_sum[w];
  L.pre[tid] = base;
  if (tid == THREADS - 1) L.pre[THREADS] = base + own;
  __syncthreads();
}

// Values that are the same in all lanes, as such.
__device__ __forceinline__ long long in_all_lanes(long long x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)x), hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
  return (long long)((uint64_t)hi << 32 | lo);
}

// Request r again: out of LDS where each thread has one.
template <int THREADS>
__device__ __forceinline__ Request request_again(const AttnArgs &a, const Line<THREADS> &L, int r) {
  if (a.R > THREADS) return request_of(a, r);
  const Request &q = L.request[r];
  return {__builtin_amdgcn_readfirstlane(q.t0), __builtin_amdgcn_readfirstlane(q.n),
          __builtin_amdgcn_readfirstlane(q.len)};
}

// A tile in the line.
struct Tile {
  Request q;
  int r, h, x;             // its request, key head, number
  int row0, rows;
  int places, blocks;      // that its rows may see: the first `places`, in `blocks` blocks
  int weight;              // Cost::weight
  long long first, after;  // its stretch of the line
  int tiles;               // of its key head
};
// The rest of a tile from q, r, h, x and first.
template <int RT, int KB, int HALF>
__device__ __forceinline__ void fill_tile(const AttnArgs &a, Tile &t, const Cost<RT, HALF> &cost) {
  t.tiles = cost.tiles;
  t.row0 = t.x * RT;
  t.rows = t.x == cost.tiles - 1 ? cost.last_rows : RT;
  t.weight = cost.weight(t.x);
  t.after = t.first + cost.of(t.x);
  t.places = t.q.len;
  if (!a.mask) t.places = min(t.q.len, max(0, t.q.len - t.q.n + node_of(a, t.row0 + t.rows - 1) + 1));
  t.blocks = t.places > 0 ? (t.places - 1) / KB + 1 : 1;
}
// The tile that place u of the line is in.
template <int RT, int KB, int HALF, int THREADS>
__device__ __forceinline__ Tile tile_at(const AttnArgs &a, const Line<THREADS> &L, long long u) {
  Tile t;
  // the last thread whose requests begin at or before it, and its request
  const int per = run_of<THREADS>(a.R);
  int run = 0, last = (a.R - 1) / per;
  while (run < last) {
    const int mid = (run + last + 1) >> 1;
    if (in_all_lanes(L.pre[mid]) <= u) run = mid;
    else last = mid - 1;
  }
  long long before = in_all_lanes(L.pre[run]);
  t.r = run * per;
  t.q = request_again(a, L, t.r);
  for (; t.r + 1 < min(a.R, run * per + per); t.r++) {
    const long long all = Cost<RT, HALF>(a, t.q).of_request(a);
    if (before + all > u) break;
    before += all;
    t.q = request_again(a, L, t.r + 1);
  }
  const Cost<RT, HALF> cost(a, t.q);
  // (the product is off by less than 1: n_heads <= 2^10)
  t.h = (int)((double)(u - before) * __builtin_amdgcn_rcp((double)cost.all));
  t.h = min(max(t.h, 0), a.c.n_heads - 1);
  if (t.h * cost.all > u - before) t.h--;
  else if ((t.h + 1) * cost.all <= u - before) t.h++;
  const long long head = before + t.h * cost.all;
  int lo = 0, hi = cost.tiles - 1;  // the last tile that begins at or before it
  while (lo < hi) {
    const int mid = lo + ((hi - lo + 1) >> 1);
    if (head + cost.of_first(mid) <= u) lo = mid;
    else hi = mid - 1;
  }
  t.x = lo;
  t.first = head + cost.of_first(lo);
  fill_tile<RT, KB, HALF>(a, t, cost);
  return t;
}
// The next tile (there is one).
template <int RT, int KB, int HALF, int THREADS>
__device__ __forceinline__ void next_tile(const AttnArgs &a, const Line<THREADS> &L, Tile &t) {
  t.first = t.after;
  if (++t.x == t.tiles) {
    t.x = 0;
    if (++t.h == a.c.n_heads) {
      t.h = 0;
      do t.q = request_again(a, L, ++t.r);
      while (t.q.n == 0 && t.r + 1 < a.R);
    }
  }
  fill_tile<RT, KB, HALF>(a, t, Cost<RT, HALF>(a, t.q));
}

// The tile's first block that is done after place u of the line (any rising
// function would do).
template <int RT, int KB>
__device__ __forceinline__ int block_from(const Tile &t, long long u) {
  if (u <= t.first) return 0;
  if (u >= t.after) return t.blocks;
  static_assert(kHalfCost == 11 && (KB & (KB - 1)) == 0, "");
  long long y = max(u - t.first - 16 * kFixedPlaces<RT>, 0ll);
  if (t.weight != 16) y = y * 93 >> 6;  // 16 / 11
  return (int)min((y + 16 * KB - 1) / (16 * KB), (long long)t.blocks);
}

// Where workgroup b's stretch of the line begins: equal ones, the last a
// little shorter.
struct Stretches {
  long long cost, each;
  __device__ __forceinline__ Stretches(const AttnArgs &a, long long cost)
      : cost(cost), each((long long)((double)cost * a.inv_groups) + (cost >> 50) + 1) {}
  __device__ __forceinline__ long long begin(int b) const { return min(cost, each * b); }
};
// Neighbours in the line read the same keys: they go to one die (workgroups
// go to the eight dies in turn, and each has an L2 of its own).
__device__ __forceinline__ int place_in_line(int b, int B) { return B % 8 ? b : (b & 7) * (B / 8) + (b >> 3); }

// ---- partial results --------------------------------------------------------

// part: for 2 B slots [part_rows][D] sums, then for each slot [part_rows]
// maxima, [part_rows] sums, then the jobs of the joining launch.
template <int D>
__device__ __forceinline__ float *part_o(const AttnArgs &a, int slot, int row) {
  return a.part + ((size_t)slot * a.part_rows + row) * D;
}
template <int D>
__device__ __forceinline__ float *part_ml(const AttnArgs &a, int B, int slot) {
  return a.part + (size_t)2 * B * a.part_rows * D + (size_t)slot * 2 * a.part_rows;
}
// What workgroup b leaves to be joined: the tile that began in its stretch and
// goes on up to workgroup `last`'s (rows = 0: none). Slots are -1 where it had
// no block.
struct JoinJob {
  int t0, h, row0, rows, last;
  int tail_slot, head_slot;  // its own part of that tile; of a tile from before its stretch
  int pad;
};
template <int D>
__device__ __forceinline__ JoinJob *join_jobs(const AttnArgs &a, int B) {
  return (JoinJob *)(a.part + (size_t)2 * B * a.part_rows * (D + 2));
}

// The walk of a workgroup over its stretch of the line, with
// segment(tile, first block, block after the last, slot or -1).
template <int RT, int KB, int HALF, int D, int THREADS, class Segment>
__device__ __forceinline__ void walk(const AttnArgs &a, Segment &&segment) {
  __shared__ Line<THREADS> L;
  line_of_tiles<RT, HALF, THREADS>(a, L);
  const int B = gridDim.x, b = place_in_line(blockIdx.x, B);
  const Stretches line(a, in_all_lanes(L.pre[THREADS]));
  const long long begin = line.begin(b), end = line.begin(b + 1);
  JoinJob job = {0, 0, 0, 0, -1, -1, -1, 0};
  Tile tile;
  for (long long u = begin; u < end;) {
    if (u == begin) tile = tile_at<RT, KB, HALF>(a, L, u);
    else next_tile<RT, KB, HALF>(a, L, tile);
    const int lo = block_from<RT, KB>(tile, u), hi = block_from<RT, KB>(tile, end);
    const int slot = lo == hi || (lo == 0 && hi == tile.blocks) ? -1 : lo ? 2 * b : 2 * b + 1;
    if (u > tile.first) job.head_slot = slot;
    else if (tile.after > end) {
      job.t0 = tile.q.t0;
      job.h = tile.h;
      job.row0 = tile.row0;
      job.rows = tile.rows;
      job.tail_slot = slot;
      int over = B;  // the first workgroup after it
      for (job.last = b; over - job.last > 1;) {
        const int mid = (job.last + over) >> 1;
        if (line.begin(mid) < tile.after) job.last = mid;
        else over = mid;
      }
    }
    if (lo < hi) segment(tile, lo, hi, slot);
    u = tile.after;
  }
  if (threadIdx.x == 0) join_jobs<D>(a, B)[b] = job;
}

// ---- numbers ----------------------------------------------------------------

// The weights are rounded to the rows' 16-bit type, since the matrix unit's fast
// products take 16-bit operands: kept in 32 bits they would be two operands
// each, and the product with the values twice as long. Each is off by at most
// half a step, independently, so that the error of an output of zero mean
// grows from its own rounding's 0.42 half steps to 0.60 (root mean square;
// bf16 1.66e-3 to 2.35e-3, fp16 2.1e-4 to 2.9e-4). Their sum is taken before
// the rounding, in fp32; scores, maxima and partial results are fp32 as well.
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
