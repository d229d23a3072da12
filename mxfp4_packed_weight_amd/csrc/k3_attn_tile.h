// Attention for many rows per key head: prompts, and trees whose nodes times
// the group's heads fill the matrix unit.
//
// The two products bound the time. A workgroup's NW waves have 32 rows each
// and share blocks of KB keys and values in LDS, two blocks in turn: while
// one is used the other arrives (16-bit caches go from memory to LDS without
// registers; e4m3 ones are widened on the way, once per workgroup), and one
// barrier per block changes them over. As in the streaming kernel all is
// transposed (lane l, c = l % 32, h = l / 32):
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

// What places outside every page read.
static __device__ const uint4 kZeroRow[256 * 2 / 16] = {};

template <int D>
constexpr int kTileKeys = D == 256 ? 32 : 64;

template <bool BF, bool F8, int D, int NW>
struct Tiled {
  static constexpr int RT = 32 * NW, KB = kTileKeys<D>, KT = KB / 32;
  static constexpr int NS = D / 16, DT = D / 32;     // steps over the head, tiles of the output
  static constexpr int ROW = 2 * D, CH = D / 8;      // a row of LDS, its chunks
  static constexpr int RPI = 64 / CH;                // rows per load of a wave
  static constexpr int RPW = KB / NW, NI = RPW / RPI;  // rows and loads of a wave
  static constexpr int kBlock = KB * ROW, kBuffer = 2 * kBlock;
  static constexpr int ES = F8 ? 1 : 2;
  static_assert(NI * RPI == RPW && NI >= 1, "");

  struct Lds {
    alignas(16) char buf[2][kBuffer];  // keys, then values
    int odd;  // a block's values held ones that are not finite
  };

  struct Wave {
    u32x4 q[NS];
    f32x16 o[DT];
    float ref, sum;  // the reference exponent, this lane's part of the sum
  };
  struct Staged {  // e4m3 rows on their way
    u32x2 k[F8 ? NI : 1], v[F8 ? NI : 1];
  };
  // A block's pages, one place per lane (blocks of 32: each place twice).
  struct Places {
    int64_t offset;
    uint64_t present;
  };

  static __device__ __forceinline__ int swizzle_k(int row) {
    return D == 64 ? (row & 7) ^ ((row >> 3) & 1) : row & 15;
  }
  static __device__ __forceinline__ int swizzle_v(int row) {
    const int r = row & 3;
    return D == 64 ? 2 * r : 2 * (2 * r ^ (r >> 1));
  }

  static __device__ __forceinline__ int table_entry(const AttnArgs &a, const int32_t *row, int p, int len) {
    if (p >= len) return -1;
    const uint32_t b = __umulhi(2u * (uint32_t)p, a.page_magic) >> a.page_shift;
    return b < (uint32_t)a.blocks ? row[b] : -1;
  }
  static __device__ __forceinline__ Places places(const AttnArgs &a, int p, int page) {
    const bool there = page >= 0 && page < a.c.n_pages;
    const uint32_t b = __umulhi(2u * (uint32_t)p, a.page_magic) >> a.page_shift;
    const int64_t at = page * a.c.page_stride + (int)((uint32_t)p - b * a.c.page_size) * a.c.slot_stride;
    return {there ? at * ES : 0, __ballot(there)};
  }

  // This wave's rows of a block: into LDS, or (e4m3) into registers.
  static __device__ __forceinline__ void fetch(const Places &pl, const char *k, const char *v, lds_char *buf, Staged &st,
                                               int lane, int wave) {
    const int pos = lane % CH;
    const bool full = pl.present == ~0ull;
#pragma unroll
    for (int i = 0; i < NI; i++) {
      const int row = wave * RPW + i * RPI + lane / CH;
      const uint32_t lo = __shfl((int)(uint32_t)pl.offset, row), hi = __shfl((int)(pl.offset >> 32), row);
      const int64_t at = (int64_t)((uint64_t)hi << 32 | lo);
      if constexpr (F8) {
        const bool there = (pl.present >> row) & 1;
        st.k[i] = *(const u32x2 *)(k + at + 8 * pos);
        st.v[i] = *(const u32x2 *)(v + at + 8 * pos);
        if (!there) st.k[i] = st.v[i] = u32x2{0, 0};
      } else {
        const int kc = 16 * (pos ^ swizzle_k(row)), vc = 16 * (pos ^ swizzle_v(row));
        const char *kp = k + at + kc, *vp = v + at + vc;
        if (!full && !((pl.present >> row) & 1)) {
          kp = (const char *)kZeroRow + kc;
          vp = (const char *)kZeroRow + vc;
        }
        lds_char *to = buf + (wave * RPW + i * RPI) * ROW;
        __builtin_amdgcn_global_load_lds((global_ptr)kp, (__attribute__((address_space(3))) void *)to, 16, 0, 0);
        __builtin_amdgcn_global_load_lds((global_ptr)vp, (__attribute__((address_space(3))) void *)(to + kBlock), 16, 0,
                                         0);
      }
    }
  }
  static __device__ __forceinline__ void put(const Staged &st, lds_char *buf, int lane, int wave) {
    if constexpr (F8) {
      const int pos = lane % CH;
      auto wide = [](u32x2 w) {
        return u32x4{widen2<BF, false>(w[0]), widen2<BF, true>(w[0]), widen2<BF, false>(w[1]), widen2<BF, true>(w[1])};
      };
#pragma unroll
      for (int i = 0; i < NI; i++) {
        const int row = wave * RPW + i * RPI + lane / CH;
        lds_char *to = buf + row * ROW;
        *(__attribute__((address_space(3))) u32x4 *)(to + 16 * (pos ^ swizzle_k(row))) = wide(st.k[i]);
        *(__attribute__((address_space(3))) u32x4 *)(to + kBlock + 16 * (pos ^ swizzle_v(row))) = wide(st.v[i]);
      }
    }
  }

  // All of this wave's copies are in and its reads are done; then all waves'.
  static __device__ __forceinline__ void change_over() {
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  // Values that are not finite numbers set to zero (0 times NaN would reach
  // rows that do not see their place).
  static __device__ __forceinline__ void make_finite(lds_char *v, int *odd) {
    bool lost = false;
    for (int x = threadIdx.x; x < kBlock / 16; x += 64 * NW) {
      auto *p = (__attribute__((address_space(3))) u32x4 *)(v + 16 * x);
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

  // The products of those values with the weights of the rows that see them.
  static __device__ __forceinline__ void add_not_finite(const AttnArgs &a, f32x16 *o, const float (*x)[16],
                                                        const uint32_t *vis, const char *v, const int32_t *table,
                                                        int k0, uint64_t present, int len, int c, int h) {
    for (int key = 0; key < KB; key++) {
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
      const int page = table_entry(a, table, k0 + key, len);
      const Places pl = places(a, k0 + key, page);
      const char *row = v + pl.offset;
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

  // One block of KB places for this wave's rows. PARTIAL: with places that
  // some rows do not see; from: the first such place.
  template <bool PARTIAL>
  static __device__ __forceinline__ void block(const AttnArgs &a, Wave &w, const Request &rq, int node, int k0,
                                               int from, uint64_t present, float scale, lds_char *buf, bool odd,
                                               const char *v, const int32_t *table, int lane) {
    typedef const __attribute__((address_space(3))) u32x4 *row_ptr;
    typedef __attribute__((address_space(3))) s16x4 *tr_ptr;
    if (PARTIAL) asm volatile("" : "+v"(lane));  // nothing of this is kept in registers outside
    const int c = lane & 31, h = lane >> 5;
    f32x16 s[KT];
    {
      const int f = h ^ swizzle_k(c);  // (the same for row c + 32)
      const lds_char *row = buf + c * ROW;
#pragma unroll
      for (int u = 0; u < KT; u++) s[u] = f32x16{};
      auto key = [&](int x) { return *(row_ptr)(row + 16 * (2 * (x / KT) ^ f) + 32 * (x % KT) * ROW); };
      constexpr int N = NS * KT, kAhead = 4;
      u32x4 k[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; x++) k[x] = key(x);
#pragma unroll
      for (int x = 0; x < N; x++) {
        __builtin_amdgcn_sched_barrier(0);  // reads stay kAhead products ahead
        s[x % KT] = mfma32<BF>(k[x % kAhead], w.q[x / KT], s[x % KT]);
        if (x + kAhead < N) k[x % kAhead] = key(x + kAhead);
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
        if (k0 + KB > from) vis[u] = seen(a, rq, node, k0 + 32 * u, vis[u]);
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
    const lds_char *row = buf + kBlock + key * ROW + 8 * (i16 & 1);
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
    if (PARTIAL && odd) add_not_finite(a, w.o, x, vis, v, table, k0, present, rq.len, c, h);
  }

  // A block is used while the next one arrives. The two buffers do not
  // overlap: reads of `cur` need not wait for the copies into `next`.
  template <bool PARTIAL>
  static __device__ __forceinline__ void step(const AttnArgs &a, Wave &w, const Request &rq, int node, int k0,
                                              int from, uint64_t present, const Places &then, bool more, bool use,
                                              float scale, lds_char *__restrict__ cur, lds_char *__restrict__ next,
                                              bool odd, const char *k, const char *v, const int32_t *table, int lane,
                                              int wave) {
    Staged st;
    if (more) fetch(then, k, v, next, st, lane, wave);
    if (use) block<PARTIAL>(a, w, rq, node, k0, from, present, scale, cur, odd, v, table, lane);
    if (F8 && more) put(st, next, lane, wave);
  }

  // A tile's blocks [lo, hi): its result, or a partial one into `slot`.
  static __device__ __forceinline__ void segment(const AttnArgs &a, Lds &L, const Tile &tile, int lo, int hi, int slot,
                                                 int B) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 31,
              h = lane >> 5;
    const Request &rq = tile.q;
    const int rows = rq.n * a.G, first_row = tile.row0 + 32 * wave, row = first_row + c;
    const bool on = row < rows, any = first_row < rows;
    const int node = on ? row / a.G : 0, hq = tile.h * a.G + (on ? row - node * a.G : 0);
    Wave w;
    // a negative scale turns the queries round, so that the largest product
    // has the largest score
    const uint32_t turn = a.scale < 0.f ? 0x80008000u : 0u;
    const uint16_t *q = a.q + (int64_t)(rq.t0 + node) * a.q_stride + hq * D + 8 * h;
#pragma unroll
    for (int s = 0; s < NS; s++) w.q[s] = on && a.scale != 0.f ? *(const u32x4 *)(q + 16 * s) ^ turn : u32x4{0, 0, 0, 0};
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
    lds_char *cur = (lds_char *)L.buf[0], *next = (lds_char *)L.buf[1];
    const int in_block = lane % KB;
    int page = table_entry(a, table, lo * KB + in_block, rq.len);
    Places now = places(a, lo * KB + in_block, page), then = now;
    page = table_entry(a, table, (lo + 1) * KB + in_block, rq.len);
    {
      Staged st;
      fetch(now, k, v, cur, st, lane, wave);
      put(st, cur, lane, wave);
    }
    // blocks below `whole` are seen by all rows, but for pages that are not there
    const int whole = min(hi, max(tile_from, 0) / KB);
    for (int j = lo; j < hi;) {
      for (; j < whole && now.present == ~0ull; j++) {
        change_over();
        const bool more = j + 1 < hi;
        if (more) {
          then = places(a, (j + 1) * KB + in_block, page);
          page = table_entry(a, table, (j + 2) * KB + in_block, rq.len);
        }
        step<false>(a, w, rq, node, j * KB, from, ~0ull, then, more, any, scale, cur, next, false, k, v, table, lane,
                    wave);
        now = then;
        lds_char *t = cur;
        cur = next;
        next = t;
      }
      if (j >= hi) break;
      const int k0 = j * KB;
      change_over();
      bool odd = false;
      if (k0 + KB > tile_from) {
        if (threadIdx.x == 0) L.odd = 0;
        change_over();
        make_finite(cur + kBlock, &L.odd);
        change_over();
        odd = L.odd != 0;
      }
      const bool more = j + 1 < hi;
      if (more) {
        then = places(a, k0 + KB + in_block, page);
        page = table_entry(a, table, k0 + 2 * KB + in_block, rq.len);
      }
      step<true>(a, w, rq, node, k0, from, now.present, then, more, k0 < until, scale, cur, next, odd, k, v, table,
                 lane, wave);
      now = then;
      lds_char *t = cur;
      cur = next;
      next = t;
      j++;
    }
    change_over();  // LDS is free for the next tile
    const float sum = sum_xor32(w.sum);
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
      float *out = part_o<RT, D>(a, slot, 32 * wave + c) + 4 * h;
#pragma unroll
      for (int t = 0; t < DT; t++)
#pragma unroll
        for (int b = 0; b < 4; b++)
          *(f32x4 *)(out + 32 * t + 8 * b) =
              f32x4{w.o[t][4 * b], w.o[t][4 * b + 1], w.o[t][4 * b + 2], w.o[t][4 * b + 3]};
      if (h == 0) {
        float *ml = part_ml<RT, D>(a, B, slot);
        ml[32 * wave + c] = w.ref;
        ml[RT + 32 * wave + c] = sum;
      }
    }
  }
};

template <bool BF, bool F8, int D, int NW>
__global__ __launch_bounds__(64 * NW, 2) void attn_tile_kernel(AttnArgs a) {
  using S = Tiled<BF, F8, D, NW>;
  extern __shared__ long long pre[];
  __shared__ typename S::Lds L;
  walk<S::RT, S::KB, D, 64 * NW>(a, pre, [&](const Tile &tile, int lo, int hi, int slot) {
    S::segment(a, L, tile, lo, hi, slot, gridDim.x);
  });
}

}  // namespace k3
