// Attention for few rows per key head: decoding, small trees.
//
// The keys and values are read once and bound the time, so they go from
// memory into registers, without shared memory or barriers on the way: each
// of a workgroup's four waves takes every fourth run of 32 places (two runs at
// once of short e4m3 rows, for as many bytes under way), and the waves'
// results meet at the tile's end. Everything is transposed, so that no
// value crosses lanes between the two products (lane l, c = l % 16, g = l / 16):
//   S^T = K Q^T   rows: 2 x 16 places, columns: 16 rows of the tile.
//                 K from memory in the operand's layout (lane: place c, 8
//                 values of the head); the result's lane holds row c of the
//                 tile and places 16 u + 4 g + 0..3.
//   O^T = V^T P^T contraction over the 32 places in any order that both
//                 operands share: element j of lane g is place
//                 16 (j / 4) + 4 g + j % 4, which is what the lane's scores
//                 are. V is read in rows (16 lanes side by side cover a row,
//                 D / 16 values each) and turned within the lane by byte
//                 permutes; product e takes value e of each lane's.
// Maximum and sum are the row's own lanes', but for two lane swaps. Only the
// maximum's large rises rescale the output (kSlack).
//
// The rows' places come from the page table one run ahead, through a few
// hundred bytes of LDS per wave.
//
// Measured: one token of each of 64 requests of up to 8191 places, 8 query heads
// to a key head, 8 key heads of 128 in bf16, 1.09 GB: 188 us, 5.8 TB/s (a plain
// read on this card reaches 7.1, a copy 5.1); in e4m3 108 us, 5.1 TB/s. 8 key
// heads of 64: 103 us, 5.3 TB/s; 4 of 256: 188 us, 5.8 TB/s.
#pragma once

#include "k3_attn.h"

namespace k3 {

constexpr int kStreamWaves = 4, kStreamThreads = 64 * kStreamWaves;
// Runs of 32 places that a wave loads at once: two of e4m3 rows where they are
// short (64 requests of up to 8191 places: 113 -> 109 us at a head of 128, 75 ->
// 68 at 64; 16-bit rows of 64 gain nothing).
template <bool F8, int D>
constexpr int kStreamRuns = F8 && D <= 128 ? 2 : 1;

// BF: bf16 (else fp16) queries, outputs and weights; F8: the cache is e4m3.
template <bool BF, bool F8, int D, int QT>
struct Stream {
  static constexpr int RT = 16 * QT, NS = D / 32, DPL = D / 16;
  static constexpr int ES = F8 ? 1 : 2;
  static constexpr int RUNS = kStreamRuns<F8, D>, PLACES = 32 * RUNS;
  static constexpr int KB = PLACES * kStreamWaves;  // a block's places
  static constexpr int VW = DPL * ES / 4;     // words of a row of V per lane
  static constexpr int KW = F8 ? 2 : 4;       // words of a K operand
  static constexpr int kPad = D + 4;
  struct Lds {
    int64_t offset[kStreamWaves][PLACES];
    float ml[kStreamWaves][2][RT];
    float o[kStreamWaves][16 * kPad];
  };

  struct Wave {
    u32x4 q[QT][NS];
    uint32_t k[RUNS][2][NS][KW];
    uint32_t v[RUNS][8][VW];
    f32x4 o[QT][DPL];
    float ref[QT], sum[QT];  // the reference exponent, this lane's part of the sum
    uint32_t present[RUNS];
  };

  // Value d of the head that element j of step s holds in lane group g.
  static __device__ __forceinline__ int d_of(int s, int g) {
    return F8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
  }

  static __device__ __forceinline__ int table_entry(const AttnArgs &a, const int32_t *row, int p, int len) {
    if (p >= len) return -1;
    const uint32_t b = __umulhi(2u * (uint32_t)p, a.page_magic) >> a.page_shift;
    return b < (uint32_t)a.blocks ? row[b] : -1;
  }

  // The places from k0 on: this lane's (lane % PLACES) page is `page`. Leaves
  // the rows' offsets in LDS; places that are not there read row 0.
  static __device__ __forceinline__ void places(const AttnArgs &a, Wave &w, int64_t *offset, int lane, int k0,
                                                int page) {
    const int p = k0 + lane % PLACES;
    const bool there = page >= 0 && page < a.c.n_pages;
    const uint32_t b = __umulhi(2u * (uint32_t)p, a.page_magic) >> a.page_shift;
    const int64_t at = page * a.c.page_stride + (int)((uint32_t)p - b * a.c.page_size) * a.c.slot_stride;
    wave_sync();  // the last run's readers are done
    if (lane < PLACES) offset[lane] = there ? at * ES : 0;
    wave_sync();
    const uint64_t all = __ballot(there);
#pragma unroll
    for (int r = 0; r < RUNS; r++) w.present[r] = (uint32_t)(all >> (32 * r));
  }

  // Keys and values are read once, so they pass the caches by (not kept there
  // for later: 5.25 -> 5.95 TB/s, 64 requests of up to 8191 places).
  template <class T>
  static __device__ __forceinline__ T read_once(const char *p) {
    return __builtin_nontemporal_load((const T *)p);
  }

  static __device__ __forceinline__ void load_k(Wave &w, const char *k, const int64_t *offset, int r, int c, int g) {
#pragma unroll
    for (int u = 0; u < 2; u++) {
      const char *p = k + offset[32 * r + 16 * u + c];
      if (F8) {
#pragma unroll
        for (int s = 0; s < NS; s += 2) {
          const u32x4 x = read_once<u32x4>(p + d_of(s, g));
          w.k[r][u][s][0] = x[0];
          w.k[r][u][s][1] = x[1];
          w.k[r][u][s + 1][0] = x[2];
          w.k[r][u][s + 1][1] = x[3];
        }
      } else {
#pragma unroll
        for (int s = 0; s < NS; s++) {
          const u32x4 x = read_once<u32x4>(p + 2 * d_of(s, g));
#pragma unroll
          for (int i = 0; i < KW; i++) w.k[r][u][s][i] = x[i];
        }
      }
    }
  }

  // Value e of those that lane c has: runs of 16 bytes, so that 16 lanes' runs
  // lie side by side.
  static constexpr int kRun = DPL < 16 / ES ? DPL : 16 / ES;
  static __device__ __forceinline__ int value_of(int c, int e) { return 16 * kRun * (e / kRun) + kRun * c + e % kRun; }

  static __device__ __forceinline__ void load_v(Wave &w, const char *v, const int64_t *offset, int r, int c, int g) {
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const char *p = v + offset[32 * r + 16 * (j / 4) + 4 * g + j % 4];
      if constexpr (VW == 1) {
        w.v[r][j][0] = read_once<uint32_t>(p + c * 4);
      } else if constexpr (VW == 2) {
        const u32x2 x = read_once<u32x2>(p + c * 8);
        w.v[r][j][0] = x[0];
        w.v[r][j][1] = x[1];
      } else {
#pragma unroll
        for (int i = 0; i < VW; i += 4) {
          const u32x4 x = read_once<u32x4>(p + 64 * i + c * 16);
#pragma unroll
          for (int e = 0; e < 4; e++) w.v[r][j][i + e] = x[e];
        }
      }
    }
  }

  static __device__ __forceinline__ void load(Wave &w, const char *k, const char *v, const int64_t *offset, int c,
                                              int g) {
#pragma unroll
    for (int r = 0; r < RUNS; r++) load_k(w, k, offset, r, c, g);
#pragma unroll
    for (int r = 0; r < RUNS; r++) load_v(w, v, offset, r, c, g);
  }

  static __device__ __forceinline__ u32x4 k_operand(const uint32_t (&k)[2][NS][KW], int u, int s) {
    if constexpr (F8)
      return u32x4{widen2<BF, false>(k[u][s][0]), widen2<BF, true>(k[u][s][0]), widen2<BF, false>(k[u][s][1]),
                   widen2<BF, true>(k[u][s][1])};
    else
      return u32x4{k[u][s][0], k[u][s][1], k[u][s][2], k[u][s][3]};
  }

  // V^T operands of the values 4 / ES that word i of the lane's row parts hold.
  template <class F>
  static __device__ __forceinline__ void v_operands(const uint32_t (&v)[8][VW], int i, F &&use) {
    if constexpr (F8) {
      uint32_t t[4][2];  // [value][places 0..3, 4..7] as four bytes
#pragma unroll
      for (int x = 0; x < 2; x++) {
        const uint32_t a = v[4 * x][i], b = v[4 * x + 1][i], c = v[4 * x + 2][i], d = v[4 * x + 3][i];
        const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x05010400), cd = __builtin_amdgcn_perm(d, c, 0x05010400);
        const uint32_t AB = __builtin_amdgcn_perm(b, a, 0x07030602), CD = __builtin_amdgcn_perm(d, c, 0x07030602);
        t[0][x] = __builtin_amdgcn_perm(cd, ab, 0x05040100);
        t[1][x] = __builtin_amdgcn_perm(cd, ab, 0x07060302);
        t[2][x] = __builtin_amdgcn_perm(CD, AB, 0x05040100);
        t[3][x] = __builtin_amdgcn_perm(CD, AB, 0x07060302);
      }
#pragma unroll
      for (int e = 0; e < 4; e++)
        use(4 * i + e, u32x4{widen2<BF, false>(t[e][0]), widen2<BF, true>(t[e][0]), widen2<BF, false>(t[e][1]),
                             widen2<BF, true>(t[e][1])});
    } else {
      u32x4 lo, hi;
#pragma unroll
      for (int x = 0; x < 4; x++) {
        lo[x] = __builtin_amdgcn_perm(v[2 * x + 1][i], v[2 * x][i], 0x05040100);
        hi[x] = __builtin_amdgcn_perm(v[2 * x + 1][i], v[2 * x][i], 0x07060302);
      }
      use(2 * i, lo);
      use(2 * i + 1, hi);
    }
  }

  // A word of V with its values that are not finite numbers set to zero.
  static __device__ __forceinline__ uint32_t finite(uint32_t w) {
    if constexpr (F8) {
      uint32_t m = 0;  // 0x7f and 0xff are NaN; there is no infinity
#pragma unroll
      for (int b = 0; b < 4; b++)
        if (((w >> (8 * b)) & 0x7f) == 0x7f) m |= 0xffu << (8 * b);
      return w & ~m;
    } else {
      return w & ~not_finite2<BF>(w);
    }
  }

  // Places that some rows see and others do not, with values that are not
  // finite: those values' products with the weights of the rows that see
  // them (0 times NaN would reach the others). p holds q-tile t's weights.
  static __device__ __forceinline__ void add_not_finite(f32x4 *o, const float *p, uint32_t vis, const char *v,
                                                     const int64_t *offset, float *scratch, int c, int g) {
#pragma unroll
    for (int j = 0; j < 8; j++) scratch[(16 * (j / 4) + 4 * g + j % 4) * 16 + c] = p[j];
    wave_sync();
    for (int key = 0; key < 32; key++) {
      if (!((vis >> key) & 1)) continue;
      const float weight = scratch[key * 16 + c];
      const char *row = v + offset[key];
#pragma unroll
      for (int r = 0; r < 4; r++)
#pragma unroll
        for (int e = 0; e < DPL; e++) {
          const int d = value_of(4 * g + r, e);
          float x;
          if (F8) {
            const uint32_t b = ((const uint8_t *)row)[d];
            x = (b & 0x7f) == 0x7f ? NAN : 0.f;
          } else {
            const uint32_t b = ((const uint16_t *)row)[d];
            x = not_finite2<BF>(b) & 0xffffu ? half_at<BF>(b, 0) : 0.f;
          }
          if (x != 0.f) o[e][r] += weight * x;
        }
    }
    wave_sync();
  }

  // One run of 32 places: scores, weights, and the weighted values.
  template <int RUN>
  static __device__ __forceinline__ void run(const AttnArgs &a, Wave &w, const Request &rq, const int *node, int k0,
                                             float scale, const char *v, const int64_t *offset, float *scratch, int c,
                                             int g) {
    f32x4 s[QT][2];
#pragma unroll
    for (int t = 0; t < QT; t++)
#pragma unroll
      for (int u = 0; u < 2; u++) s[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NS; i++)
#pragma unroll
      for (int u = 0; u < 2; u++) {
        const u32x4 k = k_operand(w.k[RUN], u, i);
#pragma unroll
        for (int t = 0; t < QT; t++) s[t][u] = mfma16<BF>(k, w.q[t][i], s[t][u]);
      }
    const uint32_t present = w.present[RUN];
    const bool drafts = k0 + 32 > rq.len - rq.n, partial = drafts || present != 0xffffffffu;
    bool odd = false;
    if (partial) {
      if (present != 0xffffffffu) {
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (!((present >> (16 * (j / 4) + 4 * g + j % 4)) & 1))
#pragma unroll
            for (int i = 0; i < VW; i++) w.v[RUN][j][i] = 0;
      }
      if (drafts) {
        uint32_t lost = 0;
#pragma unroll
        for (int j = 0; j < 8; j++)
#pragma unroll
          for (int i = 0; i < VW; i++) {
            const uint32_t f = finite(w.v[RUN][j][i]);
            lost |= f ^ w.v[RUN][j][i];
            w.v[RUN][j][i] = f;
          }
        odd = __ballot(lost != 0) != 0;
      }
    }
    u32x4 p[QT];
#pragma unroll
    for (int t = 0; t < QT; t++) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; j++) x[j] = s[t][j / 4][j % 4] * scale;
      uint32_t vis = 0xffffffffu;
      if (partial) {
        vis = drafts ? seen(a, rq, node[t], k0, present) : present;
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (!((vis >> (16 * (j / 4) + 4 * g + j % 4)) & 1)) x[j] = -INFINITY;
      }
      float top = x[0];
#pragma unroll
      for (int j = 1; j < 8; j++) top = fmaxf(top, x[j]);
      if (__ballot(top > w.ref[t] + (kLift<BF> + kSlack))) {
        top = max_xor16(max_xor32(top)) - kLift<BF>;
        const float ref = fmaxf(w.ref[t], top);
        const float keep = w.ref[t] == ref ? 1.f : exp2_hw(w.ref[t] - ref);
        w.ref[t] = ref;
        w.sum[t] *= keep;
#pragma unroll
        for (int e = 0; e < DPL; e++) w.o[t][e] *= keep;
      }
      const float ref = w.ref[t] == -INFINITY ? 0.f : w.ref[t];
      float part = 0.f;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        x[j] = exp2_hw(x[j] - ref);
        part += x[j];
      }
      w.sum[t] += part;
#pragma unroll
      for (int i = 0; i < 4; i++) p[t][i] = pack2<BF>(x[2 * i], x[2 * i + 1]);
      if (odd) add_not_finite(w.o[t], x, vis, v, offset, scratch, c, g);
    }
#pragma unroll
    for (int i = 0; i < VW; i++)
      v_operands(w.v[RUN], i, [&](int e, u32x4 operand) {
#pragma unroll
        for (int t = 0; t < QT; t++) w.o[t][e] = mfma16<BF>(operand, p[t], w.o[t][e]);
      });
  }

  // A tile's blocks [lo, hi): its result, or a partial one into `slot`.
  static __device__ __forceinline__ void segment(const AttnArgs &a, Lds &L, const Tile &tile, int lo, int hi,
                                                 int slot, int B) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, g = lane >> 4;
    const Request &rq = tile.q;
    const int rows = rq.n * a.G;
    Wave w;
    int node[QT];
#pragma unroll
    for (int t = 0; t < QT; t++) {
      const int row = tile.row0 + 16 * t + c;
      const bool on = row < rows;
      const int i = on ? node_of(a, row) : 0, hq = tile.h * a.G + (on ? row - i * a.G : 0);
      node[t] = i;
      const uint16_t *q = a.q + (rq.t0 + i) * a.q_stride + hq * D;
#pragma unroll
      for (int s = 0; s < NS; s++) w.q[t][s] = on ? *(const u32x4 *)(q + d_of(s, g)) : u32x4{0, 0, 0, 0};
      w.ref[t] = -INFINITY;
      w.sum[t] = 0.f;
#pragma unroll
      for (int e = 0; e < DPL; e++) w.o[t][e] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const float scale = a.scale * (a.c.k_scale ? a.c.k_scale[tile.h] : 1.f) * kLog2e;
    const char *k = (const char *)a.c.k + tile.h * a.c.head_stride * ES;
    const char *v = (const char *)a.c.v + tile.h * a.c.head_stride * ES;
    const int32_t *table = a.table + (size_t)tile.r * a.blocks;
    int64_t *offset = L.offset[wave];
    const int end = (int)min((long long)hi * KB, (long long)tile.places);
    int k0 = lo * KB + PLACES * wave;
    int page = table_entry(a, table, k0 + lane % PLACES, rq.len);
    if (k0 < end) {
      places(a, w, offset, lane, k0, page);
      load(w, k, v, offset, c, g);
      page = table_entry(a, table, k0 + KB + lane % PLACES, rq.len);
      for (; k0 < end; k0 += KB) {
        run<0>(a, w, rq, node, k0, scale, v, offset, L.o[wave], c, g);
        if (RUNS > 1 && k0 + 32 < end)
          run<RUNS - 1>(a, w, rq, node, k0 + 32, scale, v, offset + PLACES - 32, L.o[wave], c, g);
        if (k0 + KB < end) {
          places(a, w, offset, lane, k0 + KB, page);
          page = table_entry(a, table, k0 + 2 * KB + lane % PLACES, rq.len);
          load(w, k, v, offset, c, g);
        }
      }
    }
    merge(a, L, w, tile, rows, slot, B);
  }

  // The four waves' results to the tile's, and out.
  static __device__ __forceinline__ void merge(const AttnArgs &a, Lds &L, Wave &w, const Tile &tile, int rows,
                                               int slot, int B) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, g = lane >> 4;
    const float v_scale = a.c.v_scale ? a.c.v_scale[tile.h] : 1.f;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < QT; t++) {
      const float sum = sum_xor16(sum_xor32(w.sum[t]));
      if (g == 0) {
        L.ml[wave][0][16 * t + c] = w.ref[t];
        L.ml[wave][1][16 * t + c] = sum;
      }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < QT; t++) {
      if (tile.row0 + 16 * t >= rows) break;  // the same for all waves
      if (t) __syncthreads();
      float ref = L.ml[0][0][16 * t + c];
      for (int i = 1; i < kStreamWaves; i++) ref = fmaxf(ref, L.ml[i][0][16 * t + c]);
      const float keep = w.ref[t] == ref ? 1.f : exp2_hw(w.ref[t] - ref);
      float *mine = L.o[wave] + c * kPad;
#pragma unroll
      for (int r = 0; r < 4; r++)
#pragma unroll
        for (int e = 0; e < DPL; e += 4) {
          const f32x4 x = {w.o[t][e][r] * keep, w.o[t][e + 1][r] * keep, w.o[t][e + 2][r] * keep,
                           w.o[t][e + 3][r] * keep};
          *(f32x4 *)(mine + value_of(4 * g + r, e)) = x;
        }
      __syncthreads();
      for (int x = tid; x < 16 * (D / 4); x += kStreamThreads) {
        const int rr = x / (D / 4), d = (x - rr * (D / 4)) * 4, row = tile.row0 + 16 * t + rr;
        if (row >= rows) continue;
        float top = L.ml[0][0][16 * t + rr];
        for (int i = 1; i < kStreamWaves; i++) top = fmaxf(top, L.ml[i][0][16 * t + rr]);
        float sum = 0.f;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < kStreamWaves; i++) {
          const float m = L.ml[i][0][16 * t + rr];
          sum += L.ml[i][1][16 * t + rr] * (m == top ? 1.f : exp2_hw(m - top));
          o += *(const f32x4 *)(L.o[i] + rr * kPad + d);
        }
        if (slot < 0) {
          const int i = node_of(a, row), hq = tile.h * a.G + row - i * a.G;
          const size_t tok = tile.q.t0 + i;
          const float f = sum == 0.f ? 0.f : v_scale / sum;
          u32x2 y = {pack2<BF>(o[0] * f, o[1] * f), pack2<BF>(o[2] * f, o[3] * f)};
          *(u32x2 *)(a.out + tok * a.out_stride + hq * D + d) = y;
          if (a.lse && d == 0) a.lse[tok * a.Hq + hq] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
        } else {
          *(f32x4 *)(part_o<D>(a, slot, 16 * t + rr) + d) = o;
          if (d == 0) {
            float *ml = part_ml<D>(a, B, slot);
            ml[16 * t + rr] = top;
            ml[a.part_rows + 16 * t + rr] = sum;
          }
        }
      }
    }
    __syncthreads();  // LDS is free for the next tile
  }
};

template <bool BF, bool F8, int D, int QT>
__global__ __launch_bounds__(kStreamThreads) void attn_stream_kernel(AttnArgs a) {
  using S = Stream<BF, F8, D, QT>;
  __shared__ typename S::Lds L;
  walk<S::RT, S::KB, 0, D, kStreamThreads>(a, [&](const Tile &tile, int lo, int hi, int slot) {
    S::segment(a, L, tile, lo, hi, slot, gridDim.x);
  });
}

}  // namespace k3
