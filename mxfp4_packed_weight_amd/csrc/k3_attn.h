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
//
// Windows. A row at position x sees the places below `sinks` and those above
// x - window. Of a tile's places only those up to the sinks' end and from its
// first row's window on are taken, in runs of 32: they are numbered without the gap, as
// if the request were so much shorter (its rows' positions and windows with
// it; what is below the gap is seen by the sinks' rule alone), and
// real_place() turns such a place into the cache's. Tiles are short then, and
// often alike: where that takes less time, workgroups get whole tiles (each
// counts as one unit of the line), and nothing is joined.
#pragma once

#include <math.h>

#include "k3_kv.h"
#include "k3_lanes.h"

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
// (With a window, tiles of blocks of 256 places count three times as much: 64
// single tokens over up to 8191 places with exponents 118 -> 110 us, 128 of them
// 217 -> 199; 512 places are no better.)
template <int RT, int KB, bool WIN>
constexpr int kFixedPlaces = RT >= 128 ? 512 : WIN && KB >= 256 ? 384 : 128;
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
// With a window a tile has at most `cap`: tiles from `capped` on. unit: what a
// tile counts if they go whole (0: they do not).
template <int RT, int KB, int HALF, bool WIN>
struct Cost {
  int tiles, last_rows;
  long long base, slope, all;
  long long cap, capped, unit;  // WIN
  static constexpr long long kFixed = 16 * kFixedPlaces<RT, KB, WIN>;
  __device__ __forceinline__ Cost(const AttnArgs &a, const Request &q, long long unit = 0) : unit(unit) {
    const long long rows = (long long)q.n * a.G;
    tiles = (int)((rows + RT - 1) / RT);
    last_rows = (int)(rows - (long long)(tiles - 1) * RT);
    const bool causal = !a.mask && q.len >= q.n;
    slope = causal ? a.slope : 0;
    base = 16ll * (causal ? q.len - q.n : q.len) + slope;
    if constexpr (WIN) {
      cap = 16ll * a.sinks + 16ll * a.window + (causal ? slope : 16ll * q.n);
      // (off by a tile or so it would do as well: every workgroup has the same)
      const double room = (double)(cap - base);
      capped = room < 0. ? 0 : !slope ? tiles : min((long long)(room * __builtin_amdgcn_rcp((double)slope)) + 1, (long long)tiles);
    }
    all = tiles ? of_first(tiles - 1) + of(tiles - 1) : 0;
  }
  // a place's cost; the first x tiles of a key head; tile x
  __device__ __forceinline__ int weight(int x) const { return x == tiles - 1 && last_rows <= HALF ? kHalfCost : 16; }
  __device__ __forceinline__ long long of_first(long long x) const {
    if constexpr (WIN) {
      if (unit) return x * unit;
      const long long y = min(x, capped);
      return x * kFixed + y * base + slope * (y * (y - 1) / 2) + (x - y) * cap;
    }
    return x * (kFixed + base) + slope * (x * (x - 1) / 2);
  }
  __device__ __forceinline__ long long of(int x) const {
    if (WIN && unit) return unit;
    const long long places = WIN && x >= capped ? cap : base + slope * x;
    return kFixed + (places * weight(x) >> 4);
  }
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

// What a tile counts if they go whole, else 0. They do if the most that a
// workgroup has then takes no longer than an equal stretch and what two parts of
// tiles cost more than whole ones (a tile's fixed cost, and about as much for the
// parts' way through memory and the joining launch). all: in sixteenths of a
// place; most: the longest tile in places.
constexpr int kUnit = 16;
template <int RT, int KB>
__device__ __forceinline__ long long unit_of(const AttnArgs &a, long long all, long long tiles, int most) {
  if (a.whole) return kUnit;
  return ceil((double)tiles * a.inv_groups) * most <= (double)all / 16 * a.inv_groups + 2 * kFixedPlaces<RT, KB, true> ? kUnit : 0;
}
template <int THREADS>
struct Counts {
  long long tiles[THREADS / 64];  // of the waves
  int most[THREADS / 64];
};
template <int RT, int KB, int HALF, bool WIN, int THREADS>
__device__ __forceinline__ long long line_of_tiles(const AttnArgs &a, Line<THREADS> &L) {
  __shared__ Counts<WIN ? THREADS : 64> counts;
  const int tid = threadIdx.x, lane = tid & 63, per = run_of<THREADS>(a.R);
  long long own = 0;
  long long own_tiles = 0;  // (cu that goes back and forth counts rows many times)
  int most = 0;
  for (int r = tid * per; r < min(a.R, tid * per + per); r++) {
    const Request q = request_of(a, r);
    const Cost<RT, KB, HALF, WIN> cost(a, q);
    own += cost.of_request(a);
    L.request[tid] = q;
    if constexpr (WIN) {
      own_tiles += (long long)cost.tiles * a.c.n_heads;
      const long long longest = cost.tiles ? max(cost.of(cost.tiles - 1), cost.of(max(cost.tiles - 2, 0))) : 0;
      most = max(most, (int)min(longest >> 4, (long long)INT32_MAX));
    }
  }
  long long incl = own, tiles = own_tiles;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const long long x = __shfl_up(incl, m);
    if (lane >= m) incl += x;
    if constexpr (WIN) {
      const long long t = __shfl_up(tiles, m);
      if (lane >= m) tiles += t;
      most = max(most, __shfl_xor(most, m));
    }
  }
  if (lane == 63) L.wave_sum[tid >> 6] = incl;
  if (WIN && lane == 63) {
    counts.tiles[tid >> 6] = tiles;
    counts.most[tid >> 6] = most;
  }
  __syncthreads();
  long long base = incl - own, unit = 0;
  for (int w = 0; w < (tid >> 6); w++) base += L.wave_sum[w];
  if constexpr (WIN) {
    long long all = 0, all_tiles = 0, before = tiles - own_tiles;
    for (int w = 0; w < THREADS / 64; w++) {
      all += L.wave_sum[w];
      if (w < (tid >> 6)) before += counts.tiles[w];
      all_tiles += counts.tiles[w];
      most = max(most, counts.most[w]);
    }
    unit = unit_of<RT, KB>(a, all, all_tiles, most);
    if (unit) {
      base = kUnit * before;
      own = kUnit * own_tiles;
    }
  }
  L.pre[tid] = base;
  if (tid == THREADS - 1) L.pre[THREADS] = base + own;
  __syncthreads();
  return unit;
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
  // WIN: places of the sinks' runs, those that are left out behind them, the
  // first place (without the gap) that is in the window of all rows
  int sinks, skipped, near;
};
// Place y of a tile's, counted without the gap, in the cache; and the request
// as it is without the gap.
template <bool WIN>
__device__ __forceinline__ int real_place(const Tile &t, int y) {
  return WIN && y >= t.sinks ? y + t.skipped : y;
}
template <bool WIN>
__device__ __forceinline__ Request without_gap(const Tile &t) {
  return {t.q.t0, t.q.n, t.q.len - (WIN ? t.skipped : 0)};
}
// What a tile's rows see, from q, row0 and rows.
template <int KB, bool WIN>
__device__ __forceinline__ void fill_places(const AttnArgs &a, Tile &t) {
  t.places = t.q.len;
  if (!a.mask) t.places = min(t.q.len, max(0, t.q.len - t.q.n + node_of(a, t.row0 + t.rows - 1) + 1));
  if constexpr (WIN) {
    // (a tree's row is at its request's last committed place or later)
    const int ctx = t.q.len - t.q.n, first = a.mask ? ctx - 1 : ctx + node_of(a, t.row0);
    t.sinks = (min(a.sinks, max(t.places, 0)) + 31) & -32;
    t.skipped = max(0, (min(max(0, first - a.window + 1), max(t.places - 1, 0)) & -32) - t.sinks);
    t.places -= t.skipped;
    t.near = t.places - a.window;
  }
  t.blocks = t.places > 0 ? (t.places - 1) / KB + 1 : 1;
}
// The rest of a tile from q, r, h, x and first.
template <int RT, int KB, int HALF, bool WIN>
__device__ __forceinline__ void fill_tile(const AttnArgs &a, Tile &t, const Cost<RT, KB, HALF, WIN> &cost) {
  t.tiles = cost.tiles;
  t.row0 = t.x * RT;
  t.rows = t.x == cost.tiles - 1 ? cost.last_rows : RT;
  t.weight = cost.weight(t.x);
  t.after = t.first + cost.of(t.x);
  fill_places<KB, WIN>(a, t);
}
// The tile that place u of the line is in.
template <int RT, int KB, int HALF, bool WIN, int THREADS>
__device__ __forceinline__ Tile tile_at(const AttnArgs &a, const Line<THREADS> &L, long long unit, long long u) {
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
    const long long all = Cost<RT, KB, HALF, WIN>(a, t.q, unit).of_request(a);
    if (before + all > u) break;
    before += all;
    t.q = request_again(a, L, t.r + 1);
  }
  const Cost<RT, KB, HALF, WIN> cost(a, t.q, unit);
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
  fill_tile<RT, KB, HALF, WIN>(a, t, cost);
  return t;
}
// The next tile (there is one).
template <int RT, int KB, int HALF, bool WIN, int THREADS>
__device__ __forceinline__ void next_tile(const AttnArgs &a, const Line<THREADS> &L, long long unit, Tile &t) {
  t.first = t.after;
  if (++t.x == t.tiles) {
    t.x = 0;
    if (++t.h == a.c.n_heads) {
      t.h = 0;
      do t.q = request_again(a, L, ++t.r);
      while (t.q.n == 0 && t.r + 1 < a.R);
    }
  }
  fill_tile<RT, KB, HALF, WIN>(a, t, Cost<RT, KB, HALF, WIN>(a, t.q, unit));
}

// The same in scalar registers: what was worked out in fp64 is in vector ones
// otherwise, of which the walk holds more than it has with a window.
__device__ __forceinline__ void to_scalars(Tile &t) {
  for (int *x : {&t.q.t0, &t.q.n, &t.q.len, &t.r, &t.h, &t.x, &t.row0, &t.rows, &t.places, &t.blocks, &t.weight,
                 &t.tiles, &t.sinks, &t.skipped, &t.near})
    *x = __builtin_amdgcn_readfirstlane(*x);
  t.first = in_all_lanes(t.first);
  t.after = in_all_lanes(t.after);
}

// The tile's first block that is done after place u of the line (any rising
// function would do).
template <int RT, int KB, bool WIN>
__device__ __forceinline__ int block_from(const Tile &t, long long u) {
  if (u <= t.first) return 0;
  if (u >= t.after) return t.blocks;
  static_assert(kHalfCost == 11 && (KB & (KB - 1)) == 0, "");
  long long y = max(u - t.first - 16 * kFixedPlaces<RT, KB, WIN>, 0ll);
  if (t.weight != 16) y = y * 93 >> 6;  // 16 / 11
  return (int)min((y + 16 * KB - 1) / (16 * KB), (long long)t.blocks);
}

// The same line where every request is one tile of each key head, which most
// calls of the streaming kernel have: a quarter of the way's instructions (each
// 128 bytes of them are fetched anew by every launch, and take longer than they
// run: one place of one request 13.7 -> 11.1 us). Says whether they are.
template <int RT, int KB>
__device__ __forceinline__ long long short_cost(const Tile &t) {
  return t.rows ? 16ll * (kFixedPlaces<RT, KB, true> + t.places) : 0;
}
__device__ __forceinline__ void as_one_tile(const AttnArgs &a, Tile &t) {
  t.x = t.row0 = 0;
  t.rows = t.q.n * a.G;
  t.weight = 16;
  t.tiles = 1;
}
template <int RT, int KB, int THREADS>
__device__ __forceinline__ bool short_line(const AttnArgs &a, Line<THREADS> &L, long long &unit) {
  __shared__ Counts<THREADS> counts;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Tile t;
  t.q = {0, 0, 0};
  if (tid < a.R) t.q = request_of(a, tid);
  as_one_tile(a, t);
  fill_places<KB, true>(a, t);
  const bool one = t.rows <= RT;
  const uint64_t here = __ballot(t.rows > 0);
  const long long own = short_cost<RT, KB>(t) * a.c.n_heads;
  long long incl = own;
  int most = t.rows ? kFixedPlaces<RT, KB, true> + t.places : 0;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const long long x = __shfl_up(incl, m);
    if (lane >= m) incl += x;
    most = max(most, __shfl_xor(most, m));
  }
  L.request[tid] = t.q;
  if (lane == 63) {
    L.wave_sum[wave] = incl;
    counts.tiles[wave] = __popcll(here);
    counts.most[wave] = most;
  }
  if (!__syncthreads_and(one)) return false;
  long long all = 0, base = incl - own;
  int tiles = 0, before = __popcll(here & ((1ull << lane) - 1));
#pragma unroll
  for (int w = 0; w < THREADS / 64; w++) {
    if (w < wave) {
      base += L.wave_sum[w];
      before += counts.tiles[w];
    }
    all += L.wave_sum[w];
    tiles += counts.tiles[w];
    most = max(most, counts.most[w]);
  }
  unit = unit_of<RT, KB>(a, all, tiles * a.c.n_heads, most);
  if (unit) {
    base = (long long)(kUnit * a.c.n_heads) * before;
    all = (long long)(kUnit * a.c.n_heads) * tiles;
  }
  L.pre[tid] = base;
  if (tid == 0) L.pre[THREADS] = all;
  __syncthreads();
  return true;
}
// The tile that place u of it is in, and the next one.
template <int RT, int KB, int THREADS>
__device__ __forceinline__ Tile short_tile_at(const AttnArgs &a, const Line<THREADS> &L, long long unit, long long u) {
  Tile t;
  int r = 0;  // requests that end at or before it
#pragma unroll
  for (int w = 0; w < THREADS; w += 64) r += __popcll(__ballot(L.pre[w + 1 + (threadIdx.x & 63)] <= u));
  t.r = r;
  t.q = request_again(a, L, r);
  as_one_tile(a, t);
  fill_places<KB, true>(a, t);
  const long long cost = unit ? unit : short_cost<RT, KB>(t), head = in_all_lanes(L.pre[r]);
  // (a quotient below 2^10, off by less than 1)
  t.h = (int)((float)(u - head) / (float)cost);
  t.h = min(max(t.h, 0), a.c.n_heads - 1);
  if (t.h * cost > u - head) t.h--;
  else if ((t.h + 1) * cost <= u - head) t.h++;
  t.first = head + t.h * cost;
  t.after = t.first + cost;
  return t;
}
template <int RT, int KB, int THREADS>
__device__ __forceinline__ void short_next_tile(const AttnArgs &a, const Line<THREADS> &L, long long unit, Tile &t) {
  if (++t.h == a.c.n_heads) {
    t.h = 0;
    do t.q = request_again(a, L, ++t.r);
    while (t.q.n == 0 && t.r + 1 < a.R);
    as_one_tile(a, t);
    fill_places<KB, true>(a, t);
  }
  t.first = t.after;
  t.after += unit ? unit : short_cost<RT, KB>(t);
}

// Where workgroup b's stretch of the line begins: equal ones, the last a
// little shorter. Whole tiles: as equal as they can be.
struct Stretches {
  long long cost, each, unit;
  double groups;  // 1 / them
  __device__ __forceinline__ Stretches(const AttnArgs &a, long long cost, long long unit)
      : cost(cost), each((long long)((double)cost * a.inv_groups) + (cost >> 50) + 1), unit(unit), groups(a.inv_groups) {}
  __device__ __forceinline__ long long begin(int b) const {
    // (the half keeps the quotient off whole numbers, where it is rounded either way)
    if (unit) return (long long)(((double)(cost / kUnit) * b + 0.5) * groups) * kUnit;
    return min(cost, each * b);
  }
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
// SHORT: with the way of its own for requests of one tile.
template <int RT, int KB, int HALF, bool WIN, bool SHORT, int D, int THREADS, class Segment>
__device__ __forceinline__ void walk(const AttnArgs &a, Segment &&segment) {
  __shared__ Line<THREADS> L;
  long long unit = 0;
  bool brief = false;
  if constexpr (SHORT) brief = a.R <= THREADS && short_line<RT, KB>(a, L, unit);
  if (!brief) unit = line_of_tiles<RT, KB, HALF, WIN, THREADS>(a, L);
  unit = WIN ? in_all_lanes(unit) : 0;
  const int B = gridDim.x, b = place_in_line(blockIdx.x, B);
  const Stretches line(a, in_all_lanes(L.pre[THREADS]), unit);
  const long long begin = line.begin(b), end = line.begin(b + 1);
  JoinJob job = {0, 0, 0, 0, -1, -1, -1, 0};
  Tile tile;
  for (long long u = begin; u < end;) {
    if (SHORT && brief) {
      if (u == begin) tile = short_tile_at<RT, KB>(a, L, unit, u);
      else short_next_tile<RT, KB>(a, L, unit, tile);
    } else if (u == begin) tile = tile_at<RT, KB, HALF, WIN>(a, L, unit, u);
    else next_tile<RT, KB, HALF, WIN>(a, L, unit, tile);
    if constexpr (WIN) to_scalars(tile);
    const int lo = block_from<RT, KB, WIN>(tile, u), hi = block_from<RT, KB, WIN>(tile, end);
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
// Two e4m3 values (exact in either 16-bit type): bytes 0, 1 or 2, 3 of w,
// times a power of two.
template <bool BF, bool HI>
__device__ __forceinline__ uint32_t widen2(uint32_t w, float power = 1.f) {
  if (BF) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, power, HI));
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, power, HI));
}
// 2^(byte - 127)
__device__ __forceinline__ float power_of(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }
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
// Of a cache with exponents: whether a code times its power, in fp32 (exact), is
// none of the finite numbers of the rows' type; with powers up to kSafePower no
// code but NaN's is.
template <bool BF>
constexpr float kSafePower = BF ? 0x1p119f : 0x1p7f;  // 448 times it is below 2^128, 65504
template <bool BF>
__device__ __forceinline__ bool past_type(float x) {
  return !(fabsf(x) < (BF ? INFINITY : 65520.f));
}
// The product if it is one of those, as the infinity or NaN it is in the type, else 0.
template <bool BF>
__device__ __forceinline__ float not_finite_product(uint32_t code, float power) {
  const float x = __builtin_amdgcn_cvt_f32_fp8((int)code, 0) * power;
  return past_type<BF>(x) ? x * INFINITY : 0.f;
}
template <bool BF>
__device__ __forceinline__ float half_at(uint32_t w, int hi) {
  if (BF) return __builtin_bit_cast(float, hi ? w & 0xffff0000u : w << 16);
  return (float)__builtin_bit_cast(f16x2, w)[hi];
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

// The first place in the window of node i (its position is its request's last
// committed place's and the nodes of its own that it sees further on).
__device__ __forceinline__ int window_of(const AttnArgs &a, const Request &q, int i) {
  int at = q.len - q.n + i;
  if (a.mask) {
    at = q.len - q.n - 1;
    const uint32_t *row = (const uint32_t *)a.mask + (size_t)(q.t0 + i) * a.words;
    for (int w = 0; w < a.words && 32 * w < q.n; w++) {
      const int left = q.n - 32 * w;
      at += __popc(left < 32 ? row[w] & ((1u << left) - 1) : row[w]);
    }
  }
  return at - a.window + 1;
}
// Of the 32 places from k0 on, those in a window from `near` on or below the sinks' end.
__device__ __forceinline__ uint32_t in_window(const AttnArgs &a, int near, int k0) {
  const int y = near - k0, z = a.sinks - k0;
  return (y <= 0 ? 0xffffffffu : y < 32 ? ~0u << y : 0u) | (z >= 32 ? 0xffffffffu : z > 0 ? (1u << z) - 1 : 0u);
}

}  // namespace k3
