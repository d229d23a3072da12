// Attention for many rows per key head: prompts, and trees whose nodes times
// the group's heads fill the matrix unit.
//
// The two products bound the time, and next to them the exponentials. Eight
// waves of 32 rows share blocks of KB keys and values in LDS. Blocks are
// fetched kAhead turns before their use, straight from memory to LDS (e4m3
// ones into a ring of their own, and widened from there one turn ahead, once
// for all waves), with one barrier per block. A tile of up to 128 rows would
// leave half of the waves without work: there, two waves share 32 rows, each
// has half of every block, and they join their results at the end.
// As in the streaming kernel all is transposed (lane l, c = l % 32, h = l / 32):
//   S^T = K Q^T   rows: 32 places, columns: the wave's 32 rows. The lane has
//                 row c's scores of places 8 b + 4 h + 0..3.
//   O^T = V^T P^T 16 places per product in the order in which the lane has
//                 their weights; V's columns come out of LDS by the
//                 transposing read, four places of one column to a lane.
// A row of LDS is cut into 16-byte chunks whose places are permuted by the
// row's number, so that the reads of 32 rows' same chunk (keys) and of four
// rows' neighbouring chunks (values) spread over the banks.
#pragma once

#include "k3_attn.h"

namespace k3 {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef const __attribute__((address_space(1))) void *global_ptr;

template <bool BF>
__device__ __forceinline__ f32x16 mfma32(u32x4 x, u32x4 y, f32x16 c) {
  if (BF)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0,
                                                   0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0,
                                                0);
}

constexpr int kAttnWaves = 8, kAttnRows = 32 * kAttnWaves, kAttnThreads = 64 * kAttnWaves;
template <int D>
constexpr int kAttnKeys = D == 256 ? 32 : 64;
// Tiles of so many rows go two waves to 32 rows (not with blocks of 32).
template <int D>
constexpr int kPairedRows = kAttnKeys<D> == 64 ? kAttnRows / 2 : 0;

template <bool BF, bool F8, int D>
struct Tiled {
  static constexpr int NW = kAttnWaves, RT = kAttnRows, KB = kAttnKeys<D>;
  static constexpr int NS = D / 16, DT = D / 32;     // steps over the head, tiles of the output
  static constexpr int ROW = 2 * D;                  // a row of LDS, D / 8 chunks
  static constexpr int ES = F8 ? 1 : 2;
  static constexpr int CH = D * ES / 16;             // chunks of a row of the cache
  static constexpr int RPL = 64 / CH;                // rows per load of a wave
  static constexpr int NL = 2 * KB / RPL / NW;       // loads of a wave, keys and values
  static constexpr int kBlock = KB * ROW, kBuffer = 2 * kBlock, kRaw = 2 * KB * D;
  static constexpr int kAhead = F8 ? 3 : 2;
  static constexpr int kBuffers = F8 ? 2 : kAhead + 1, kRaws = F8 ? kAhead : 0;
  static constexpr int kInFlight = (F8 ? kAhead - 2 : kAhead - 1) * NL;
  static constexpr int kListed = 64;                 // blocks in the list of rows
  static_assert(NL >= 1 && NL * NW * RPL == 2 * KB, "");

  struct Lds {
    alignas(16) char buf[kBuffers * kBuffer + kRaws * kRaw];  // blocks: keys, then values
    int64_t row[kListed * KB];  // where the places' rows are, of 64 blocks in turn
    uint64_t present[kListed];  // which places of a block are there
    int odd;                    // a block's values held ones that are not finite
  };

  struct Wave {
    u32x4 q[NS];
    f32x16 o[DT];
    float ref, sum;  // the reference exponent, this lane's part of the sum
  };
  static __device__ __forceinline__ int swizzle_k(int row) {
    return D == 64 ? (row & 7) ^ ((row >> 3) & 1) : row & 15;
  }
  static __device__ __forceinline__ int swizzle_v(int row) {
    const int r = row & 3;
    return D == 64 ? 2 * r : 2 * (2 * r ^ (r >> 1));
  }

  // Byte offset of a place's row; -1 if it has no page.
  static __device__ __forceinline__ int64_t place(const AttnArgs &a, const int32_t *table, int p, int end) {
    if (p >= end) return -1;
    const uint32_t b = __umulhi(2u * (uint32_t)p, a.page_magic) >> a.page_shift;
    const int page = b < (uint32_t)a.blocks ? table[b] : -1;
    if (page < 0 || page >= a.c.n_pages) return -1;
    return (page * a.c.page_stride + (int)((uint32_t)p - b * a.c.page_size) * a.c.slot_stride) * ES;
  }
  // Lists half of the 64 blocks, from block x on, and says which of them have
  // places that are not there (their rows are read from the cache's first).
  static __device__ __forceinline__ uint64_t list(const AttnArgs &a, Lds &L, const int32_t *table, int x, int end,
                                                  uint64_t holes) {
    const int at = x % kListed;
#pragma unroll
    for (int i = 0; i < kListed / 2 * KB / kAttnThreads; i++) {
      const int n = i * kAttnThreads + threadIdx.x;
      const int64_t row = place(a, table, x * KB + n, end);
      L.row[at * KB + n] = row < 0 ? 0 : row;
      const uint64_t there = __ballot(row >= 0);
      const int lane = n & 63;
      if (KB == 64 && lane == 0) L.present[at + n / KB] = there;
      if (KB == 32 && lane % 32 == 0) L.present[at + n / KB] = there >> lane | 0xffffffff00000000ull;
    }
    __syncthreads();
    const uint64_t mine = __ballot(L.present[at + threadIdx.x % (kListed / 2)] != ~0ull) & 0xffffffffu;
    return (holes & ~(0xffffffffull << at)) | mine << at;
  }

  // A copy of 16 bytes per lane from memory to LDS, in order from `to` on. The
  // compiler is not to know: it would have every read of LDS wait for it.
  // change_over() is what waits.
  static __device__ __forceinline__ void copy(const char *from, lds_char *to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)to)), "v"(from)
                 : "memory");
  }
  // This wave's loads of block x.
  static __device__ __forceinline__ void fetch(const Lds &L, int x, const char *k, const char *v, lds_char *to,
                                               uint32_t lane, int wave) {
    const uint32_t pos = lane % CH, sub = lane / CH;
    const int64_t *rows = L.row + x % kListed * KB + sub;
#pragma unroll
    for (int i = 0; i < NL; i++) {
      const bool values = NL > 1 ? i & 1 : wave >= NW / 2;
      const int group = NL > 1 ? wave * (NL / 2) + i / 2 : wave % (NW / 2), first = group * RPL;
      // (the swizzles are linear in the bits of the row)
      const int chunk = F8 ? 16 * pos
                           : values ? 16 * (pos ^ swizzle_v(sub)) ^ 16 * swizzle_v(first)
                                    : 16 * (pos ^ swizzle_k(sub)) ^ 16 * swizzle_k(first);
      copy((values ? v : k) + rows[first] + chunk, to + (values ? KB * CH * 16 : 0) + group * 1024);
    }
  }
  // A block of e4m3 rows from LDS into LDS.
  static __device__ __forceinline__ void widen(const lds_char *from, lds_char *to) {
    auto wide = [](uint32_t x, uint32_t y) {
      return u32x4{widen2<BF, false>(x), widen2<BF, true>(x), widen2<BF, false>(y), widen2<BF, true>(y)};
    };
#pragma unroll
    for (int i = 0; i < kRaw / 16 / kAttnThreads; i++) {
      const int x = i * kAttnThreads + threadIdx.x;  // a chunk: two of the wide row
      const int row = x / CH, chunk = 2 * (x % CH);
      const u32x4 w = *(const __attribute__((address_space(3))) u32x4 *)(from + 16 * x);
      const int f = row < KB ? swizzle_k(row) : swizzle_v(row);
      *(__attribute__((address_space(3))) u32x4 *)(to + row * ROW + 16 * (chunk ^ f)) = wide(w[0], w[1]);
      *(__attribute__((address_space(3))) u32x4 *)(to + row * ROW + 16 * ((chunk + 1) ^ f)) = wide(w[2], w[3]);
    }
  }

  // All but the newest IN_FLIGHT of this wave's copies are in and its LDS
  // accesses are done; then all waves'.
  template <int IN_FLIGHT>
  static __device__ __forceinline__ void change_over() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(IN_FLIGHT) : "memory");
  }

  // Values at places that are not there, and those that are not finite
  // numbers, set to zero (0 times NaN would reach rows that do not see them).
  static __device__ __forceinline__ void make_finite(lds_char *v, uint64_t present, int *odd) {
    bool lost = false;
    for (uint32_t x = threadIdx.x; x < kBlock / 16; x += kAttnThreads) {
      auto *p = (__attribute__((address_space(3))) u32x4 *)(v + 16 * x);
      if (!((present >> (x / (ROW / 16))) & 1)) {
        *p = u32x4{0, 0, 0, 0};
        continue;
      }
      u32x4 w = *p;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint32_t bad = not_finite2<BF>(w[i]);
        m |= bad;
        w[i] &= ~bad;
      }
      if (m) {
        *p = w;
        lost = true;
      }
    }
    if (lost) *odd = 1;
  }

  // The products of those values with the weights of the rows that see them;
  // KT tiles of 32 places from k0 on.
  template <int KT>
  static __device__ __forceinline__ void add_not_finite(const AttnArgs &a, f32x16 *o, const float (*x)[16],
                                                        const uint32_t *vis, const char *v, const int32_t *table,
                                                        int k0, uint64_t present, int c, int h) {
    for (int key = 0; key < 32 * KT; key++) {
      if (!((present >> key) & 1)) continue;
      const int at = (key >> 5) * 16 + ((key >> 3) & 3) * 4 + (key & 3);
      float mine = 0.f;
#pragma unroll
      for (int i = 0; i < 16 * KT; i++)
        if (i == at) mine = x[i / 16][i % 16];
      const float weight = __shfl(mine, c + 32 * ((key >> 2) & 1));
      uint32_t word = vis[0];
      if (KT > 1 && key >= 32) word = vis[KT - 1];
      const bool sees = (word >> (key & 31)) & 1;
      const char *row = v + place(a, table, k0 + key, INT32_MAX);
#pragma unroll
      for (int t = 0; t < DT; t++)
#pragma unroll
        for (int i = 0; i < 16; i++) {
          const int d = 32 * t + 8 * (i / 4) + 4 * h + i % 4;
          float y;
          if (F8) {
            y = (((const uint8_t *)row)[d] & 0x7f) == 0x7f ? NAN : 0.f;
          } else {
            const uint32_t w = ((const uint16_t *)row)[d];
            y = not_finite2<BF>(w) & 0xffffu ? half_at<BF>(w, 0) : 0.f;
          }
          if (sees && y != 0.f) o[t][i] += weight * y;
        }
    }
  }

  // KT tiles of 32 places, from k0 on, for this wave's rows; keys: their rows
  // in LDS. PARTIAL: with places that some rows do not see; from: the first
  // such place.
  template <bool PARTIAL, int KT>
  static __device__ __forceinline__ void block(const AttnArgs &a, Wave &w, const Request &rq, int node, int k0,
                                               int from, uint64_t present, float scale, lds_char *keys, bool odd,
                                               const char *v, const int32_t *table, uint32_t lane) {
    typedef const __attribute__((address_space(3))) u32x4 *row_ptr;
    typedef __attribute__((address_space(3))) s16x4 *tr_ptr;
    if (PARTIAL) asm volatile("" : "+v"(lane));  // nothing of this is kept in registers outside
    const int c = lane & 31, h = lane >> 5;
    f32x16 s[KT];
    {
      const int f = h ^ swizzle_k(c);  // (the same for row c + 32)
      const lds_char *row = keys + c * ROW;
#pragma unroll
      for (int u = 0; u < KT; u++) s[u] = f32x16{};
      auto key = [&](int x) { return *(row_ptr)(row + 16 * (2 * (x / KT) ^ f) + 32 * (x % KT) * ROW); };
      constexpr int N = NS * KT, kReads = 4;
      u32x4 k[kReads];
#pragma unroll
      for (int x = 0; x < kReads; x++) k[x] = key(x);
#pragma unroll
      for (int x = 0; x < N; x++) {
        __builtin_amdgcn_sched_barrier(0);  // reads stay kReads products ahead
        s[x % KT] = mfma32<BF>(k[x % kReads], w.q[x / KT], s[x % KT]);
        if (x + kReads < N) k[x % kReads] = key(x + kReads);
      }
    }
    float x[KT][16];
    uint32_t vis[KT];
#pragma unroll
    for (int u = 0; u < KT; u++) {
#pragma unroll
      for (int i = 0; i < 16; i++) x[u][i] = s[u][i];
      if (PARTIAL) {
        vis[u] = (uint32_t)(present >> (32 * u));
        if (k0 + 32 * KT > from) vis[u] = seen(a, rq, node, k0 + 32 * u, vis[u]);
#pragma unroll
        for (int i = 0; i < 16; i++)
          if (!((vis[u] >> (8 * (i / 4) + 4 * h + i % 4)) & 1)) x[u][i] = -INFINITY;
      }
    }
    float top = x[0][0];
#pragma unroll
    for (int u = 0; u < KT; u++)
#pragma unroll
      for (int i = 0; i < 16; i++) top = fmaxf(top, x[u][i]);
    top *= scale;
    if (__ballot(top > w.ref + (kLift<BF> + kSlack))) {
      top = max_xor32(top) - kLift<BF>;
      const float ref = fmaxf(w.ref, top);
      const float keep = w.ref == ref ? 1.f : exp2_hw(w.ref - ref);
      w.ref = ref;
      w.sum *= keep;
#pragma unroll
      for (int t = 0; t < DT; t++) w.o[t] *= keep;
    }
    const float ref = w.ref == -INFINITY ? 0.f : w.ref;
    // lane i of a group of 16 reads row i / 4's values 4 (i % 4) + 0..3 of the
    // group's 4 x 16 and receives column i's
    const int i16 = lane & 15, key = 4 * h + i16 / 4, f = swizzle_v(key);
    const lds_char *row = keys + kBlock + key * ROW + 8 * (i16 & 1);
    auto value = [&](int j, int t) {  // places 16 j + 0..15, tile t of the head
      const lds_char *at = row + 16 * ((4 * t + 2 * ((lane >> 4) & 1) + ((i16 >> 1) & 1)) ^ f) + 16 * j * ROW;
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)at));
      const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)(at + 8 * ROW)));
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    // weight i of the 8 that product j takes from this lane
    float part[2] = {0.f, 0.f};
    auto weight = [&](int j, int i, u32x4 &p) {
      float *y = &x[j / 2][8 * (j & 1)];
      y[i] = exp2_hw(fmaf(y[i], scale, -ref));
      part[i & 1] += y[i];
      if (i & 1) p[i / 2] = pack2<BF>(y[i - 1], y[i]);
    };
    constexpr int J = 2 * KT;
    u32x4 p[2], vt[DT];
#pragma unroll
    for (int t = 0; t < DT; t++) vt[t] = value(0, t);
#pragma unroll
    for (int i = 0; i < 8; i++) weight(0, i, p[0]);
    // the products of one step beside the reads and the exponentials of the
    // next, in this order
#pragma unroll
    for (int j = 0; j < J; j++)
#pragma unroll
      for (int t = 0; t < DT; t++) {
        __builtin_amdgcn_sched_barrier(0);
        w.o[t] = mfma32<BF>(vt[t], p[j & 1], w.o[t]);
        if (j + 1 < J) {
          vt[t] = value(j + 1, t);
#pragma unroll
          for (int i = 8 * t / DT; i < 8 * (t + 1) / DT; i++) weight(j + 1, i, p[(j + 1) & 1]);
        }
      }
    __builtin_amdgcn_sched_barrier(0);
    w.sum += part[0] + part[1];
    if (PARTIAL && odd) add_not_finite<KT>(a, w.o, x, vis, v, table, k0, present, c, h);
  }

  // A tile's blocks [lo, hi): its result, or a partial one into `slot`.
  // PAIRED: two waves for 32 rows, half of each block to each.
  template <bool PAIRED>
  static __device__ __forceinline__ void segment(const AttnArgs &a, Lds &L, const Tile &tile, int lo, int hi, int slot,
                                                 int B) {
    const uint32_t lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Request &rq = tile.q;
    const int first_in_tile = 32 * (PAIRED ? wave >> 1 : wave), in_tile = first_in_tile + (int)c;
    const int rows = rq.n * a.G, first_row = tile.row0 + first_in_tile, row = tile.row0 + in_tile;
    const bool on = row < rows, any = first_row < rows;
    const int node = on ? row / a.G : 0, hq = tile.h * a.G + (on ? row - node * a.G : 0);
    Wave w;
    // a negative scale turns the queries round, so that the largest product
    // has the largest score
    const uint32_t round = a.scale < 0.f ? 0x80008000u : 0u;
    const uint16_t *q = a.q + (int64_t)(rq.t0 + node) * a.q_stride + hq * D + 8 * h;
#pragma unroll
    for (int s = 0; s < NS; s++)
      w.q[s] = on && a.scale != 0.f ? *(const u32x4 *)(q + 16 * s) ^ round : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < DT; t++) w.o[t] = f32x16{};
    w.ref = -INFINITY;
    w.sum = 0.f;
    const float k_scale = a.c.k_scale ? a.c.k_scale[tile.h] : 1.f;
    const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale) * k_scale * kLog2e;
    const char *k = (const char *)a.c.k + tile.h * a.c.head_stride * ES;
    const char *v = (const char *)a.c.v + tile.h * a.c.head_stride * ES;
    const int32_t *table = a.table + (size_t)tile.r * a.blocks;
    // places from here on: some rows of the tile (of this wave) do not see them; none of the wave's does
    const int ctx = rq.len - rq.n;
    const int tile_from = a.mask ? ctx : ctx + tile.row0 / a.G + 1;
    const int from = a.mask || !any ? ctx : ctx + first_row / a.G + 1;
    const int until = !any ? 0 : a.mask ? rq.len : ctx + (min(first_row + 31, rows - 1)) / a.G + 1;
    const int end = min(hi * KB, rq.len);
    constexpr int KT = PAIRED ? 1 : KB / 32;
    const int half = PAIRED ? 32 * (wave & 1) : 0;
    lds_char *buf = (lds_char *)L.buf, *ring = buf + kBuffers * kBuffer;
    int cur = 0, raw = 0;  // the block in use, the ring's place that is fetched into
    uint64_t holes = 0;    // blocks of the list with places that are not there
    // Fetches block x and returns where the block to use is.
    auto advance = [&](int x) {
      lds_char *now = buf + cur * kBuffer;
      if constexpr (F8) {
        fetch(L, x, k, v, ring + raw * kRaw, lane, wave);
        raw = raw + 1 == kRaws ? 0 : raw + 1;
        widen(ring + raw * kRaw, buf + (1 - cur) * kBuffer);  // the oldest in the ring: the next to use
        cur = 1 - cur;
      } else {
        fetch(L, x, k, v, buf + (cur == 0 ? kBuffers - 1 : cur - 1) * kBuffer, lane, wave);
        cur = cur + 1 == kBuffers ? 0 : cur + 1;
      }
      return now;
    };
    holes = list(a, L, table, lo & -(kListed / 2), end, holes);
    for (int j = lo - kAhead; j < hi; j++) {
      // blocks that all rows see whole
      if (j >= lo) {
        const int next = (j + kAhead + kListed / 2 - 1) & -(kListed / 2);  // block to list from
        const int whole = min(min(hi, max(tile_from, 0) / KB), next - kAhead);
        for (; j < whole && !((holes >> (j % kListed)) & 1); j++) {
          change_over<kInFlight>();
          lds_char *now = advance(j + kAhead);
          if (any)
            block<false, KT>(a, w, rq, node, 0, 0, ~0ull, scale, now + half * ROW, false, v, table, lane);
        }
        if (j >= hi) break;
      }
      const int k0 = j * KB;
      change_over<kInFlight>();
      if ((j + kAhead) % (kListed / 2) == 0 && j + kAhead > lo)
        holes = list(a, L, table, j + kAhead, end, holes);
      lds_char *now = advance(j + kAhead);
      if (j < lo) continue;
      const uint64_t present = in_all_lanes(L.present[j % kListed]);
      bool odd = false;
      if (k0 + KB > tile_from || present != ~0ull) {
        if (threadIdx.x == 0) L.odd = 0;
        change_over<63>();
        make_finite(now + kBlock, present, &L.odd);
        change_over<63>();
        odd = L.odd != 0;
      }
      if (k0 + half < until)
        block<true, KT>(a, w, rq, node, k0 + half, from, present >> half, scale, now + half * ROW, odd, v, table,
                        lane);
    }
    change_over<0>();  // LDS is free
    float sum = sum_xor32(w.sum);
    if constexpr (PAIRED) {
      float *theirs = (float *)L.buf + (wave >> 1) * (16 * DT + 2) * 64 + (int)lane;
      if (wave & 1) {
#pragma unroll
        for (int t = 0; t < DT; t++)
#pragma unroll
          for (int i = 0; i < 16; i++) theirs[64 * (16 * t + i)] = w.o[t][i];
        theirs[64 * 16 * DT] = w.ref;
        theirs[64 * (16 * DT + 1)] = sum;
      }
      __syncthreads();
      if (!(wave & 1)) {
        const float m = theirs[64 * 16 * DT], top = fmaxf(w.ref, m);
        const float mine = w.ref == top ? 1.f : exp2_hw(w.ref - top), other = m == top ? 1.f : exp2_hw(m - top);
        sum = sum * mine + theirs[64 * (16 * DT + 1)] * other;
        w.ref = top;
#pragma unroll
        for (int t = 0; t < DT; t++)
#pragma unroll
          for (int i = 0; i < 16; i++) w.o[t][i] = w.o[t][i] * mine + theirs[64 * (16 * t + i)] * other;
      }
      __syncthreads();
      if (wave & 1) return;
    }
    if (!on) return;
    if (slot < 0) {
      const float f = sum == 0.f ? 0.f : (a.c.v_scale ? a.c.v_scale[tile.h] : 1.f) / sum;
      const size_t tok = rq.t0 + node;
      uint16_t *out = a.out + tok * a.out_stride + hq * D + 4 * h;
#pragma unroll
      for (int t = 0; t < DT; t++)
#pragma unroll
        for (int b = 0; b < 4; b++)
          *(u32x2 *)(out + 32 * t + 8 * b) = u32x2{pack2<BF>(w.o[t][4 * b] * f, w.o[t][4 * b + 1] * f),
                                                   pack2<BF>(w.o[t][4 * b + 2] * f, w.o[t][4 * b + 3] * f)};
      if (a.lse && h == 0) a.lse[tok * a.Hq + hq] = sum == 0.f ? -INFINITY : (w.ref + log2f(sum)) * kLn2;
    } else {
      float *out = part_o<D>(a, slot, in_tile) + 4 * h;
#pragma unroll
      for (int t = 0; t < DT; t++)
#pragma unroll
        for (int b = 0; b < 4; b++)
          *(f32x4 *)(out + 32 * t + 8 * b) =
              f32x4{w.o[t][4 * b], w.o[t][4 * b + 1], w.o[t][4 * b + 2], w.o[t][4 * b + 3]};
      if (h == 0) {
        float *ml = part_ml<D>(a, B, slot);
        ml[in_tile] = w.ref;
        ml[a.part_rows + in_tile] = sum;
      }
    }
  }
};

template <bool BF, bool F8, int D>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_tile_kernel(AttnArgs a) {
  using S = Tiled<BF, F8, D>;
  __shared__ typename S::Lds L;
  walk<S::RT, S::KB, kPairedRows<D>, D, kAttnThreads>(a, [&](const Tile &tile, int lo, int hi, int slot) {
    if (kPairedRows<D> && tile.rows <= kPairedRows<D>) S::template segment<true>(a, L, tile, lo, hi, slot, gridDim.x);
    else S::template segment<false>(a, L, tile, lo, hi, slot, gridDim.x);
  });
}

}  // namespace k3
