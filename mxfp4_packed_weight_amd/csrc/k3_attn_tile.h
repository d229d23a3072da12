// Attention for many rows per key head: prompts, and trees whose nodes times
// the group's heads fill the matrix unit.
//
// The two products bound the time, and next to them the exponentials. Eight
// waves of 32 rows share blocks of KB keys and values in LDS. A wave's turn
// has two phases, one of products (the weights of the last block with its
// values, then this block's keys with the queries) and one of arithmetic (the
// scores' maximum, exponentials and sum). The two waves of a SIMD are a phase
// apart, so that the matrix unit has the one's products while the vector unit
// has the other's exponentials; a barrier per phase keeps them so. Blocks are
// fetched kAhead turns before their use, straight from memory to LDS (e4m3
// ones into a ring of their own, and widened from there one turn ahead, once
// for all waves). A tile of up to 128 rows would leave half of the waves
// without work: there, two waves share 32 rows, each has half of every block,
// and they join their results at the end. A head of 256 needs the registers of
// two waves: four waves, each with a SIMD to itself, whose products run beside
// its own exponentials.
// As in the streaming kernel all is transposed (lane l, c = l % 32, h = l / 32):
//   S^T = K Q^T   rows: 32 places, columns: the wave's 32 rows. The lane has
//                 row c's scores of places 8 b + 4 h + 0..3.
//   O^T = V^T P^T 16 places per product in the order in which the lane has
//                 their weights; V's columns come out of LDS by the
//                 transposing read, four places of one column to a lane.
// A row of LDS is cut into 16-byte chunks whose places are permuted by the
// row's number, so that the reads of 32 rows' same chunk (keys) and of four
// rows' neighbouring chunks (values) spread over the banks (no conflicts
// counted in 16-bit caches).
//
// Measured on 32 requests of 256 rows over 8192 places, 8 key heads of 128,
// bf16: 306 us (898 TFLOP/s, 3.6 TB/s), 252 us (1090 TFLOP/s) where the pages
// are few and stay in the caches; a large product of the library reaches 1227.
// What made it: reads four products ahead and in program order (390 -> 354 us),
// copies two turns ahead and no registers on the way (354 -> 337; three turns
// are no faster), the two phases (337 -> 312), products before arithmetic at
// issue (309 -> 305). Beside products the vector unit's own instructions run
// at about half their rate, exponentials freely, so that a phase is bound by
// both units together. Two waves to 32 rows: 250 -> 227 us at 128 rows.
// Heads of 256, 128 rows: 650 TFLOP/s at 5.2 TB/s, 904 with few pages.
#pragma once

#include <type_traits>

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

template <int D>
constexpr int kAttnWaves = D == 256 ? 4 : 8;
template <int D>
constexpr int kAttnThreads = 64 * kAttnWaves<D>;
template <int D>
constexpr int kAttnKeys = D == 256 ? 32 : 64;
// Tiles of so many rows go two waves to 32 rows (not with blocks of 32).
template <int D>
constexpr int kPairedRows = D == 256 ? 0 : 128;

template <bool BF, bool F8, int D>
struct Tiled {
  static constexpr int NW = kAttnWaves<D>, RT = 32 * NW, KB = kAttnKeys<D>, kThreads = kAttnThreads<D>;
  static constexpr bool kPhases = NW == 8;           // two waves to a SIMD, a phase apart
  static constexpr int NS = D / 16, DT = D / 32;     // steps over the head, tiles of the output
  static constexpr int ROW = 2 * D;                  // a row of LDS, D / 8 chunks
  static constexpr int ES = F8 ? 1 : 2;
  static constexpr int CH = D * ES / 16;             // chunks of a row of the cache
  static constexpr int RPL = 64 / CH;                // rows per load of a wave
  static constexpr int NL = 2 * KB / RPL / NW;       // loads of a wave, keys and values
  static constexpr int NR = (NL + 1) / 2;            // rows of a lane in them
  static constexpr int kBlock = KB * ROW, kBuffer = 2 * kBlock, kRaw = 2 * KB * D;
  static constexpr int kAhead = F8 ? 3 : 2;
  static constexpr int kBuffers = F8 ? 2 : kAhead + 1, kRaws = F8 ? kAhead : 0;
  static constexpr int kInFlight = (F8 ? kAhead - 2 : kAhead - 1) * NL;
  static constexpr int kListed = KB == 128 ? 32 : 64;  // blocks in the list of rows
  static_assert(NL >= 1 && NL * NW * RPL == 2 * KB, "");

  struct Lds {
    alignas(16) char buf[kBuffers * kBuffer + kRaws * kRaw];  // keys of a block, values of the one before
    int64_t row[kListed * KB];  // where the places' rows are, of kListed blocks in turn
    uint32_t present[kListed * KB / 32];  // which places of a block are there
    int odd;                    // values that are not finite were set to zero
  };

  template <int KT>
  struct Wave {
    u32x4 q[NS];
    f32x16 s[KT];     // the block's scores
    u32x4 p[2 * KT];  // its weights
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

  static __device__ __forceinline__ uint32_t block_of(const AttnArgs &a, int p) {
    return __umulhi(2u * (uint32_t)p, a.page_magic) >> a.page_shift;
  }
  // Byte offset of the row of place p, whose page (block b) is `page`; -1 if
  // there is no such page.
  static __device__ __forceinline__ int64_t row_of(const AttnArgs &a, int p, uint32_t b, int page) {
    if (page < 0 || page >= a.c.n_pages) return -1;
    return (page * a.c.page_stride + (int)((uint32_t)p - b * a.c.page_size) * a.c.slot_stride) * ES;
  }
  // Lists half of kListed blocks, from block x on, and says which of them have
  // places that are not there (their rows are read from the cache's first).
  static __device__ __forceinline__ uint64_t list(const AttnArgs &a, Lds &L, const int32_t *table, int x, int end,
                                                  uint64_t holes) {
    const int at = x % kListed;
    constexpr int N = kListed / 2 * KB / kThreads;
    int page[N];  // (all loads at once: the table has at least one entry)
#pragma unroll
    for (int i = 0; i < N; i++)
      page[i] = table[min(block_of(a, x * KB + i * kThreads + threadIdx.x), (uint32_t)a.blocks - 1)];
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int n = i * kThreads + threadIdx.x, p = x * KB + n;
      const int64_t row = p < end ? row_of(a, p, block_of(a, p), page[i]) : -1;
      L.row[at * KB + n] = row < 0 ? 0 : row;
      const uint64_t there = __ballot(row >= 0);
      if (n % 32 == 0) L.present[at * (KB / 32) + n / 32] = (uint32_t)(there >> (n & 32));
    }
    __syncthreads();
    bool hole = false;
#pragma unroll
    for (int u = 0; u < KB / 32; u++)
      hole |= L.present[(at + threadIdx.x % (kListed / 2)) * (KB / 32) + u] != 0xffffffffu;
    constexpr uint64_t kHalf = (1ull << kListed / 2) - 1;
    return (holes & ~(kHalf << at)) | (__ballot(hole) & kHalf) << at;
  }

  // A copy of 16 bytes per lane from memory to LDS, in order from `to` on. The
  // compiler is not to know: it would have every read of LDS wait for it.
  // change_over() is what waits.
  static __device__ __forceinline__ void copy(const char *from, lds_char *to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)to)), "v"(from)
                 : "m0", "memory");
  }
  // Where the rows are that a wave loads in a turn: keys of block x, values of
  // block x - 1 (the first turn has none: block `lo`, which is listed).
  struct Rows {
    int64_t key[NR], value[NR];
  };
  static __device__ __forceinline__ const int64_t *listed(const Lds &L, int x, int i, uint32_t lane, int wave) {
    const int group = NL > 1 ? wave * NR + i : wave % (NW / 2);
    return L.row + x % kListed * KB + group * RPL + lane / CH;
  }
  static __device__ __forceinline__ Rows rows_of(const Lds &L, int x, int lo, uint32_t lane, int wave) {
    Rows r;
#pragma unroll
    for (int i = 0; i < NR; i++) {
      r.key[i] = *listed(L, x, i, lane, wave);
      r.value[i] = *listed(L, max(x - 1, lo), i, lane, wave);
    }
    return r;
  }
  // (block x may not be listed yet: then these rows are not used)
  static __device__ __forceinline__ Rows rows_after(const Lds &L, const Rows &now, int x, uint32_t lane, int wave) {
    Rows r;
#pragma unroll
    for (int i = 0; i < NR; i++) {
      r.key[i] = *listed(L, x, i, lane, wave);
      r.value[i] = now.key[i];
    }
    return r;
  }
  static __device__ __forceinline__ void fetch(const Rows &r, const char *k, const char *v, lds_char *to, uint32_t lane,
                                               int wave) {
    const uint32_t pos = lane % CH, sub = lane / CH;
#pragma unroll
    for (int i = 0; i < NL; i++) {
      const bool values = NL > 1 ? i & 1 : wave >= NW / 2;
      const int group = NL > 1 ? wave * NR + i / 2 : wave % (NW / 2), first = group * RPL;
      // (the swizzles are linear in the bits of the row)
      const int chunk = F8 ? 16 * pos
                           : values ? 16 * (pos ^ swizzle_v(sub)) ^ 16 * swizzle_v(first)
                                    : 16 * (pos ^ swizzle_k(sub)) ^ 16 * swizzle_k(first);
      copy((values ? v + r.value[i / 2] : k + r.key[i / 2]) + chunk, to + (values ? KB * CH * 16 : 0) + group * 1024);
    }
  }
  // A block of e4m3 rows from LDS into LDS.
  static __device__ __forceinline__ void widen(const lds_char *from, lds_char *to) {
    auto wide = [](uint32_t x, uint32_t y) {
      return u32x4{widen2<BF, false>(x), widen2<BF, true>(x), widen2<BF, false>(y), widen2<BF, true>(y)};
    };
#pragma unroll
    for (int i = 0; i < kRaw / 16 / kThreads; i++) {
      const int x = i * kThreads + threadIdx.x;  // a chunk: two of the wide row
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
  static __device__ __forceinline__ void make_finite(lds_char *v, const uint32_t *present, int *odd) {
    bool lost = false;
    for (uint32_t x = threadIdx.x; x < kBlock / 16; x += kThreads) {
      auto *p = (__attribute__((address_space(3))) u32x4 *)(v + 16 * x);
      const uint32_t row = x / (ROW / 16);
      if (!((present[row / 32] >> row % 32) & 1)) {
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

  // Those values, at the places [p, end), to the rows that see them: whatever
  // their weights were, the sums are then no finite numbers either.
  static __device__ __forceinline__ void add_not_finite(const AttnArgs &a, f32x16 *o, const Request &rq, int node,
                                                        const char *v, const int32_t *table, int p, int end, int h) {
    for (; p < end; p++) {
      const uint32_t b = block_of(a, p);
      const int64_t at = row_of(a, p, b, table[b]);
      if (at < 0 || !(seen(a, rq, node, p, 1) & 1)) continue;
      const char *row = v + at;
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
          o[t][i] += y;
        }
    }
  }

  // Reads of operands from a turn's keys and values.
  template <int KT>
  struct Reader {
    const lds_char *keys, *vals;
    int fk, fv, column;
    __device__ __forceinline__ Reader(const lds_char *buf, uint32_t lane) {
      const int c = lane & 31, h = lane >> 5;
      keys = buf + c * ROW;
      fk = h ^ swizzle_k(c);  // (the same for rows c + 32 u)
      // lane i of a group of 16 reads row i / 4's values 4 (i % 4) + 0..3 of the
      // group's 4 x 16 and receives column i's
      const int i16 = lane & 15, row = 4 * h + i16 / 4;
      vals = buf + kBlock + row * ROW + 8 * (i16 & 1);
      fv = swizzle_v(row);
      column = 2 * ((lane >> 4) & 1) + ((i16 >> 1) & 1);
    }
    // step x / KT over the head, 32 places from 32 (x % KT) on
    __device__ __forceinline__ u32x4 key(int x) const {
      typedef const __attribute__((address_space(3))) u32x4 *ptr;
      return *(ptr)(keys + 16 * (2 * (x / KT) ^ fk) + 32 * (x % KT) * ROW);
    }
    // places 16 (x / DT) + 0..15, tile x % DT of the head
    __device__ __forceinline__ u32x4 value(int x) const {
      typedef __attribute__((address_space(3))) s16x4 *ptr;
      const lds_char *at = vals + 16 * ((4 * (x % DT) + column) ^ fv) + 16 * (x / DT) * ROW;
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)at));
      const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(at + 8 * ROW)));
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  };
  static constexpr int kReads = 4;  // products that the reads are ahead
  template <int KT>
  static __device__ __forceinline__ void scores_of(Wave<KT> &w, const Reader<KT> &in, u32x4 *k) {
    constexpr int N = NS * KT;
#pragma unroll
    for (int u = 0; u < KT; u++) w.s[u] = f32x16{};
#pragma unroll
    for (int x = 0; x < N; x++) {
      __builtin_amdgcn_sched_barrier(0);
      w.s[x % KT] = mfma32<BF>(k[x % kReads], w.q[x / KT], w.s[x % KT]);
      if (x + kReads < N) k[x % kReads] = in.key(x + kReads);
    }
  }

  // The phase of products: `values`: O += P V of the last block, `scores`:
  // S = K Q of this one. buf: the wave's part of the turn's keys and values.
  template <int KT>
  static __device__ __forceinline__ void products(Wave<KT> &w, const lds_char *buf, bool values, bool scores,
                                                  uint32_t lane) {
    const Reader<KT> in(buf, lane);
    constexpr int N = DT * 2 * KT;
    u32x4 k[kReads], vt[kReads];
    if (kPhases) __builtin_amdgcn_s_setprio(1);
    if (values) {
#pragma unroll
      for (int x = 0; x < kReads; x++) vt[x] = in.value(x);
    }
#pragma unroll
    for (int x = 0; x < kReads; x++) k[x] = in.key(x);
    if (values) {
#pragma unroll
      for (int x = 0; x < N; x++) {
        __builtin_amdgcn_sched_barrier(0);
        w.o[x % DT] = mfma32<BF>(vt[x % kReads], w.p[x / DT], w.o[x % DT]);
        if (x + kReads < N) vt[x % kReads] = in.value(x + kReads);
      }
    }
    if (scores) scores_of<KT>(w, in, k);
    if (kPhases) __builtin_amdgcn_s_setprio(0);
  }

  // The scores of places that a row does not see, to minus infinity; from: the
  // first place that some rows do not see.
  template <int KT>
  static __device__ __forceinline__ void hide(const AttnArgs &a, f32x16 *s, const Request &rq, int node, int k0,
                                              int from, const uint32_t *present, uint32_t lane) {
    const int h = lane >> 5;
#pragma unroll
    for (int u = 0; u < KT; u++) {
      uint32_t vis = present[u];
      if (k0 + 32 * KT > from) vis = seen(a, rq, node, k0 + 32 * u, vis);
      vis >>= 4 * h;
#pragma unroll
      for (int i = 0; i < 16; i++)
        if (!((vis >> (8 * (i / 4) + i % 4)) & 1)) s[u][i] = -INFINITY;
    }
  }

  // The reference exponent for the new scores; true if it rose (in any lane),
  // and `keep`, what the old sums are worth then.
  template <int KT>
  static __device__ __forceinline__ bool raise(Wave<KT> &w, float scale, float &keep) {
    float top = w.s[0][0];
#pragma unroll
    for (int u = 0; u < KT; u++)
#pragma unroll
      for (int i = 0; i < 16; i++) top = fmaxf(top, w.s[u][i]);
    top *= scale;
    if (!__ballot(top > w.ref + (kLift<BF> + kSlack))) return false;
    top = max_xor32(top) - kLift<BF>;
    const float ref = fmaxf(w.ref, top);
    keep = w.ref == ref ? 1.f : exp2_hw(w.ref - ref);
    w.ref = ref;
    return true;
  }
  // Weight i of the lane's, and its part in the sum.
  template <int KT>
  static __device__ __forceinline__ void weight(Wave<KT> &w, u32x4 *p, int i, float scale, float ref, float *part) {
    f32x16 &x = w.s[i / 16];
    x[i % 16] = exp2_hw(fmaf(x[i % 16], scale, -ref));
    part[i & 1] += x[i % 16];
    if (i & 1) p[i / 8][i % 8 / 2] = pack2<BF>(x[i % 16 - 1], x[i % 16]);
  }

  // The phase of arithmetic: the scores become weights.
  template <int KT>
  static __device__ __forceinline__ void weights(Wave<KT> &w, float scale) {
    float keep;
    if (raise<KT>(w, scale, keep)) {
      w.sum *= keep;
#pragma unroll
      for (int t = 0; t < DT; t++) w.o[t] *= keep;
    }
    const float ref = w.ref == -INFINITY ? 0.f : w.ref;
    float part[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16 * KT; i++) weight<KT>(w, w.p, i, scale, ref, part);
    w.sum += part[0] + part[1];
  }

  // Both, for a wave that has its SIMD to itself: this block's scores, then
  // the last block's values beside this one's exponentials.
  template <int KT>
  static __device__ __forceinline__ void both(Wave<KT> &w, const lds_char *buf, float scale, uint32_t lane) {
    const Reader<KT> in(buf, lane);
    u32x4 k[kReads], vt[kReads], p[2 * KT];
#pragma unroll
    for (int x = 0; x < kReads; x++) k[x] = in.key(x);
    scores_of<KT>(w, in, k);
#pragma unroll
    for (int x = 0; x < kReads; x++) vt[x] = in.value(x);
    float keep, part[2] = {0.f, 0.f};
    const bool rose = raise<KT>(w, scale, keep);
    const float ref = w.ref == -INFINITY ? 0.f : w.ref;
    constexpr int N = DT * 2 * KT, kEach = 16 * KT / N;
    static_assert(kEach >= 1, "");
#pragma unroll
    for (int x = 0; x < N; x++) {
      __builtin_amdgcn_sched_barrier(0);
      w.o[x % DT] = mfma32<BF>(vt[x % kReads], w.p[x / DT], w.o[x % DT]);
      if (x + kReads < N) vt[x % kReads] = in.value(x + kReads);
#pragma unroll
      for (int i = 0; i < kEach; i++) weight<KT>(w, p, kEach * x + i, scale, ref, part);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (rose) {
      w.sum *= keep;
#pragma unroll
      for (int t = 0; t < DT; t++) w.o[t] *= keep;
    }
    w.sum += part[0] + part[1];
#pragma unroll
    for (int i = 0; i < 2 * KT; i++) w.p[i] = p[i];
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
    const int node = on ? node_of(a, row) : 0, hq = tile.h * a.G + (on ? row - node * a.G : 0);
    constexpr int KT = PAIRED ? KB / 64 : KB / 32;
    Wave<KT> w;
    // a negative scale turns the queries round, so that the largest product
    // has the largest score; at 0 every product is 0
    const float factor = a.scale * (a.c.k_scale ? a.c.k_scale[tile.h] : 1.f) * kLog2e;
    const uint32_t round = factor < 0.f ? 0x80008000u : 0u;
    const float scale = factor == 0.f ? 1.f : fabsf(factor);
    const uint16_t *q = a.q + (int64_t)(rq.t0 + node) * a.q_stride + hq * D + 8 * h;
#pragma unroll
    for (int s = 0; s < NS; s++)
      w.q[s] = on && factor != 0.f ? *(const u32x4 *)(q + 16 * s) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < DT; t++) w.o[t] = f32x16{};
    w.ref = -INFINITY;
    w.sum = 0.f;
    const char *k = (const char *)a.c.k + tile.h * a.c.head_stride * ES;
    const char *v = (const char *)a.c.v + tile.h * a.c.head_stride * ES;
    const int32_t *table = a.table + (size_t)tile.r * a.blocks;
    // places from here on: some rows of the tile (of this wave) do not see them; none of the wave's does
    const int ctx = rq.len - rq.n;
    const int tile_from = a.mask ? ctx : ctx + node_of(a, tile.row0) + 1;
    const int from = a.mask || !any ? ctx : ctx + node_of(a, first_row) + 1;
    const int until = !any ? 0 : a.mask ? rq.len : ctx + node_of(a, min(first_row + 31, rows - 1)) + 1;
    const int end = min(hi * KB, rq.len);
    const int half = PAIRED ? 32 * KT * (wave & 1) : 0, late_wave = kPhases && wave >= NW / 2;
    lds_char *buf = (lds_char *)L.buf, *ring = buf + kBuffers * kBuffer;
    int cur = 0, raw = 0;  // the turn's buffer, the ring's place that is fetched into
    if (threadIdx.x == 0) L.odd = 0;
    uint64_t holes = list(a, L, table, lo & -(kListed / 2), end, 0);  // blocks with places that are not there
#pragma unroll
    for (int s = 0; s < NS; s++) w.q[s] ^= round;  // (only here are they waited for)
    // Begins turn j: fetches `rows` for a later one, and says where this one's
    // keys and values are, and the next one's.
    auto begin = [&](const Rows &rows, const lds_char *&now, lds_char *&next) {
      now = buf + cur * kBuffer + half * ROW;
      if constexpr (F8) {
        fetch(rows, k, v, ring + raw * kRaw, lane, wave);
        raw = raw + 1 == kRaws ? 0 : raw + 1;
        cur = 1 - cur;
        next = buf + cur * kBuffer;
        widen(ring + raw * kRaw, next);  // the oldest in the ring
      } else {
        fetch(rows, k, v, buf + (cur == 0 ? kBuffers - 1 : cur - 1) * kBuffer, lane, wave);
        cur = cur + 1 == kBuffers ? 0 : cur + 1;
        next = buf + cur * kBuffer;
      }
    };
    auto hole = [&](int j) { return (holes >> (j % kListed)) & 1; };
    auto whole = [&](int j) { return j * KB + KB <= tile_from && !hole(j); };
    // The turns from j on whose block, and the one before, all rows see whole.
    auto hot = [&](int j, auto late) {
      const int next_list = (j + kAhead + kListed / 2 - 1) & -(kListed / 2);
      const int stop = min(min(hi, max(tile_from, 0) / KB), next_list - kAhead);
      Rows rows = rows_of(L, j + kAhead, lo, lane, wave);
      for (; j < stop && !hole(j); j++) {
        const lds_char *now;
        lds_char *next;
        change_over<kInFlight>();
        begin(rows, now, next);
        rows = rows_after(L, rows, j + 1 + kAhead, lane, wave);
        if constexpr (!kPhases) {
          if (any) both<KT>(w, now, scale, lane);
          continue;
        }
        if (any) {
          if constexpr (late) weights<KT>(w, scale);
          else products<KT>(w, now, true, true, lane);
        }
        change_over<63>();
        if (any) {
          if constexpr (late) products<KT>(w, now, true, true, lane);
          else weights<KT>(w, scale);
        }
      }
      return j;
    };
    auto turns = [&](auto late) {
      for (int j = lo - kAhead; j <= hi; j++) {
        if (j > lo && whole(j - 1)) {
          j = hot(j, late);
        }
        // any other turn
        uint32_t l = lane;
        asm volatile("" : "+v"(l));  // nothing of this is kept in registers outside
        const lds_char *now;
        lds_char *next;
        change_over<kInFlight>();
        if ((j + kAhead) % (kListed / 2) == 0 && j + kAhead > lo) holes = list(a, L, table, j + kAhead, end, holes);
        begin(rows_of(L, j + kAhead, lo, lane, wave), now, next);
        if (j < lo) continue;
        if (j < hi && !whole(j)) {
          change_over<F8 ? 63 : NL>();
          make_finite(next + kBlock, L.present + j % kListed * (KB / 32), &L.odd);
          change_over<63>();
        }
        auto use = [&](int j) { return j >= lo && j < hi && j * KB + half < until; };
        for (int phase = 0; phase < 2; phase++) {
          if (phase && kPhases) change_over<63>();
          const int of = late && !phase ? j - 1 : j;  // whose arithmetic
          if (phase == late) products<KT>(w, now, use(j - 1), use(j), l);
          else if (use(of)) {
            if (!whole(of))
              hide<KT>(a, w.s, rq, node, of * KB + half, from, L.present + (of % kListed * KB + half) / 32, l);
            weights<KT>(w, scale);
          }
        }
      }
    };
    if (late_wave) turns(std::integral_constant<bool, kPhases>{});
    else turns(std::false_type{});
    const bool odd = L.odd != 0;
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
    if (odd) add_not_finite(a, w.o, rq, node, v, table, lo * KB, end, h);
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
__global__ __launch_bounds__(kAttnThreads<D>, kAttnWaves<D> / 4) void attn_tile_kernel(AttnArgs a) {
  using S = Tiled<BF, F8, D>;
  __shared__ typename S::Lds L;
  walk<S::RT, S::KB, kPairedRows<D>, D, kAttnThreads<D>>(a, [&](const Tile &tile, int lo, int hi, int slot) {
    if constexpr (kPairedRows<D> > 0) {
      if (tile.rows <= kPairedRows<D>) return S::template segment<true>(a, L, tile, lo, hi, slot, gridDim.x);
    }
    S::template segment<false>(a, L, tile, lo, hi, slot, gridDim.x);
  });
}

}  // namespace k3
