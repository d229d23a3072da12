// Log probabilities of given tokens, entropy, and the largest logits of rows.
//
//   z = beta x / ln 2,  lse / ln 2 = log2 sum 2^z,  log2 p = z - log2 sum 2^z,
//   entropy / ln 2 = log2 S - Q / S,  S = sum 2^d, Q = sum 2^d d,
//   d = z - r for the reference r = z of m,
// where m is at least near the largest of what was read so far: one pass, S and Q
// are scaled when m rises. d is one fused operation, exact but for its own rounding
// if r is taken as it was rounded. Where |r| reaches 2^20, so that what this
// rounding leaves of z of m is no longer small, d is (x - m) beta / ln 2. In 2^d d
// a d of -inf counts as the lowest number, times 0; rows without a list do that only
// in runs where the plain sum is not a number (16 bits: 56 -> 51 us with the fused
// operation). Lanes join by one change of reference each, to the largest of all, then
// plain sums (51 -> 49; 64 rows with 20 alternatives 21 -> 18).
//
// A row's logits go to the waves in runs of 64 lanes x 16. Each wave keeps the
// k <= 64 largest of its logits sorted in its lanes, one a lane. The logits of a
// run that are above the k-th are collected in LDS, and when 64 are there they are
// sorted and joined with the list: a comparison of one list with the other turned
// round leaves the largest 64 of both, six steps of sorting order them. (Putting
// them in one by one took four times as long: 64 rows of 131072 logits with 20
// alternatives 41 -> 24, now 18 us.) Until a wave has k, a run's threshold is the k-th
// largest of its lanes' own maxima.
//
// 1000 rows of 150001 fp32 logits, 600 MB: 90 us, 6.7 TB/s (a plain read reaches
// 7.1); with 20 alternatives 96 us. Rows of 16 bits are bound by the vector unit
// (ten instructions to a logit, one of them an exponential at a quarter of the
// rate): 51 us, 5.9 TB/s, 73 with 20 alternatives. One row of 131072: 10 to 11 us, two
// launches' latency; 64 rows with 20 alternatives 18 us. Runs further ahead than the
// next change nothing.
#include <math.h>

#include <algorithm>

#include "k3_lanes.h"
#include "k3_rows.h"
#include "k3_step.h"

namespace k3 {

namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves, kJoinWaves = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.4028234663852886e38f;

template <int TYPE>
constexpr int kPer = TYPE == K3_F32 ? 4 : 8;  // values of 16 bytes
template <int TYPE>
constexpr int kLoads = 16 / kPer<TYPE>;  // of a lane in a run
constexpr int kRun = 64 * 16;            // values of a run

template <int TYPE>
__device__ __forceinline__ float value_at(const void *row, int64_t i) {
  if (TYPE == K3_F32) return ((const float *)row)[i];
  const uint16_t u = ((const uint16_t *)row)[i];
  if (TYPE == K3_BF16) return __builtin_bit_cast(float, (uint32_t)u << 16);
  return (float)__builtin_bit_cast(_Float16, u);
}
template <int TYPE>
__device__ __forceinline__ void unpack(const uint4 &p, float *f) {
  if constexpr (TYPE == K3_F32) {
    f[0] = __builtin_bit_cast(float, p.x);
    f[1] = __builtin_bit_cast(float, p.y);
    f[2] = __builtin_bit_cast(float, p.z);
    f[3] = __builtin_bit_cast(float, p.w);
  } else {
    unpack8<TYPE == K3_BF16>(p, f);
  }
}

// ---- sums ---------------------------------------------------------------------

constexpr float kPlain = 0x1p20f;
// d of x for the reference m, r = m b2 rounded.
__device__ __forceinline__ float above(float x, float m, float r, float b2) {
  return fabsf(r) < kPlain ? fmaf(x, b2, -r) : (x - m) * b2;
}

struct Sums {
  float m, s, q;
  // what r's rounding left
  static __device__ __forceinline__ float rest(float m, float b2) { return above(m, m, m * b2, b2); }
  // what is known of values below a higher reference, seen from it (b2 = beta / ln 2)
  __device__ __forceinline__ void raise(float top, float b2) {
    const float fall = m == top ? 0.f : (m - top) * b2 + (rest(top, b2) - rest(m, b2));
    const float f = __builtin_amdgcn_exp2f(fall);
    q = f == 0.f ? 0.f : f * (q + fall * s);
    s *= f;
    m = top;
  }
  __device__ __forceinline__ void join(Sums o, float b2) {
    const float top = o.m > m ? o.m : m;
    raise(top, b2);
    o.raise(top, b2);
    s += o.s;
    q += o.q;
  }
  // of LANES lanes that follow one another, in each of them
  template <int LANES = 64>
  __device__ __forceinline__ void join_lanes(float b2) {
    float top = m;
    halving<LANES / 2>([&](auto d) { top = fmaxf(top, lane_xor<decltype(d)::value>(top)); });
    raise(top, b2);
    halving<LANES / 2>([&](auto d) {
      s += lane_xor<decltype(d)::value>(s);
      q += lane_xor<decltype(d)::value>(q);
    });
  }
};

// ---- lists of the largest -------------------------------------------------------

// A logit and its index as one number, larger for what comes first: greater
// values, of equal ones the lower index.
typedef uint64_t Entry;
// Rising integers for rising floats (no NaN), and back.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __builtin_bit_cast(float, u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ Entry entry_of(float v, int at) {
  return (uint64_t)ordered(v + 0.f) << 32 | ~(uint32_t)at;  // (no -0)
}
constexpr Entry kNone = (uint64_t)0x007fffffu << 32;  // -inf, index -1
__device__ __forceinline__ float value_of(Entry e) { return from_ordered((uint32_t)(e >> 32)); }
__device__ __forceinline__ int index_of(Entry e) { return (int)~(uint32_t)e; }

template <int D>
__device__ __forceinline__ Entry entry_xor(Entry x) {
  return (uint64_t)lane_xor<D>((uint32_t)(x >> 32)) << 32 | lane_xor<D>((uint32_t)x);
}
// Lane l and l ^ D in order: the larger to the lane with bit D clear, or set.
template <int D>
__device__ __forceinline__ Entry ordered_pair(Entry x, bool upper) {
  const Entry o = entry_xor<D>(x);
  return (o > x) != upper ? o : x;
}
// A list of any 64 entries, largest first.
__device__ __forceinline__ Entry sorted(Entry x, int lane) {
  x = ordered_pair<1>(x, (lane ^ lane >> 1) & 1);
  auto stage = [&](auto n) {
    constexpr int N = decltype(n)::value;
    halving<N / 2>([&](auto d) {
      constexpr int D = decltype(d)::value;
      x = ordered_pair<D>(x, !(lane & D) != !(lane & N));
    });
  };
  stage(std::integral_constant<int, 4>{});
  stage(std::integral_constant<int, 8>{});
  stage(std::integral_constant<int, 16>{});
  stage(std::integral_constant<int, 32>{});
  stage(std::integral_constant<int, 64>{});
  return x;
}
// The largest 64 of two lists.
__device__ __forceinline__ Entry joined(Entry x, Entry y, int lane) {
  const Entry o = __shfl(y, 63 - lane);
  if (o > x) x = o;
  halving<32>([&](auto d) {
    constexpr int D = decltype(d)::value;
    x = ordered_pair<D>(x, lane & D);
  });
  return x;
}
// The largest float below the k-th largest of the lanes' (no NaN), or -inf.
__device__ __forceinline__ float below_kth(float x, int k) {
  const uint32_t u = ordered(x);
  uint32_t kth = 0;
#pragma unroll
  for (int b = 31; b >= 0; b--) {
    const uint32_t with = kth | 1u << b;
    if ((int)__popcll(__ballot(u >= with)) >= k) kth = with;
  }
  // one step down; past zero's two signs
  const float v = from_ordered(kth);
  if (v == 0.f) return -0x1p-149f;
  return v == -INFINITY ? v : from_ordered(kth - 1);
}

// ---- one part of a row ------------------------------------------------------------

// A wave's loads of a run: values that are not in the row are -inf.
template <int TYPE>
__device__ __forceinline__ void load(const char *row, int V, int first, int lane, uint4 *out) {
  constexpr int PER = kPer<TYPE>, ES = 16 / PER;
#pragma unroll
  for (int i = 0; i < kLoads<TYPE>; i++) {
    const int at = first + (i * 64 + lane) * PER;
    if (at >= 0 && at <= V - PER) {
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      const u32x4 w = __builtin_nontemporal_load((const u32x4 *)(row + (int64_t)at * ES));  // (read once)
      out[i] = uint4{w[0], w[1], w[2], w[3]};
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        if (TYPE == K3_F32) {
          w[j] = at + j >= 0 && at + j < V ? ((const uint32_t *)row)[at + j] : 0xff800000u;
        } else {
          constexpr uint32_t kMinusInf = TYPE == K3_BF16 ? 0xff80u : 0xfc00u;
          const int x = at + 2 * j;
          const uint32_t lo = x >= 0 && x < V ? ((const uint16_t *)row)[x] : kMinusInf;
          const uint32_t hi = x + 1 >= 0 && x + 1 < V ? ((const uint16_t *)row)[x + 1] : kMinusInf;
          w[j] = lo | hi << 16;
        }
      }
      out[i] = uint4{w[0], w[1], w[2], w[3]};
    }
  }
}

template <int TYPE, bool TOP>
struct Wave {
  Sums sums;
  Entry list;
  float last;   // what a logit must be above to be collected
  int waiting;  // collected: in LDS, fewer than 64 between runs

  // The 64 oldest that wait (or all) into the list.
  __device__ __forceinline__ void take(Entry *wait, int lane) {
    wave_sync();
    const Entry x = lane < waiting ? wait[lane] : kNone, rest = wait[64 + lane];
    wave_sync();
    wait[lane] = rest;
    waiting = max(waiting - 64, 0);
    list = joined(list, sorted(x, lane), lane);
  }

  __device__ __forceinline__ void run(const uint4 *in, int first, float b2, int k, int lane, Entry *wait) {
    constexpr int PER = kPer<TYPE>, LOADS = kLoads<TYPE>;
    float x[LOADS][PER], most[LOADS], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < LOADS; i++) {
      unpack<TYPE>(in[i], x[i]);
      most[i] = -INFINITY;
#pragma unroll
      for (int j = 0; j < PER; j++) most[i] = fmaxf(most[i], x[i][j]);
      top = fmaxf(top, most[i]);
    }
    if (__ballot((top - sums.m) * b2 > 1.f)) sums.raise(fmaxf(sums.m, top), b2);
    const float r = sums.m * b2;
    if (!__ballot(!(fabsf(r) < kPlain))) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < LOADS; i++)
#pragma unroll
        for (int j = 0; j < PER; j++) {
          const float d = fmaf(x[i][j], b2, -r), e = __builtin_amdgcn_exp2f(d);
          sums.s += e;
          q = fmaf(e, TOP ? fmaxf(d, kLowest) : d, q);
        }
      if (!TOP && __ballot(q != q)) {  // (0 times -inf is none; with a list there are no registers for this)
        q = 0.f;
#pragma unroll
        for (int i = 0; i < LOADS; i++)
#pragma unroll
          for (int j = 0; j < PER; j++) {
            const float d = fmaf(x[i][j], b2, -r);
            q = fmaf(__builtin_amdgcn_exp2f(d), fmaxf(d, kLowest), q);
          }
      }
      sums.q += q;
    } else {
      // some lanes' at least (those that have read nothing but -inf have the lowest number's): above(), lane by lane
      const bool plain = fabsf(r) < kPlain;
      const float from = plain ? 0.f : sums.m, less = plain ? r : 0.f;
#pragma unroll
      for (int i = 0; i < LOADS; i++)
#pragma unroll
        for (int j = 0; j < PER; j++) {
          const float d = fmaf(x[i][j] - from, b2, -less), e = __builtin_amdgcn_exp2f(d);
          sums.s += e;
          sums.q = fmaf(e, fmaxf(d, kLowest), sums.q);
        }
    }
    if (!TOP) return;
    if (last == -INFINITY) last = below_kth(top, k);  // (fewer than k so far)
    // (`last` stays as it is meanwhile: these are not in the order of their indices)
    bool grown = false;
#pragma unroll
    for (int i = 0; i < LOADS; i++) {
      if (!__ballot(most[i] > last)) continue;
#pragma unroll
      for (int j = 0; j < PER; j++) {
        const bool mine = x[i][j] > last;
        const uint64_t lanes = __ballot(mine);
        if (!lanes) continue;
        const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(lanes >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)lanes, 0));
        if (mine) wait[waiting + before] = entry_of(x[i][j], first + (i * 64 + lane) * PER + j);
        waiting += (int)__popcll(lanes);
        if (waiting >= 64) {
          take(wait, lane);
          grown = true;
        }
      }
    }
    if (grown) {
      const uint32_t kth = __builtin_amdgcn_readlane((uint32_t)(list >> 32), k - 1);
      last = fmaxf(last, from_ordered(kth));
    }
  }
};

// The logit of the row's token (read long before it is used): -inf for one
// that is none.
template <int TYPE>
__device__ __forceinline__ float logit_of(const LogprobArgs &a, int t) {
  const int token = a.logprob ? a.tokens[t] : -1;
  return token >= 0 && token < a.V ? value_at<TYPE>(a.logits, t * a.stride + token) : -INFINITY;
}

template <int TYPE>
__device__ void finish(const LogprobArgs &a, int t, float logit, Sums sums, Entry list, int lane) {
  const char *row = (const char *)a.logits + t * a.stride * (16 / kPer<TYPE>);
  const float log2_s = log2f(sums.s), b2 = a.beta * kLog2e, r = sums.m * b2;
  auto log_p = [&](float x) {  // S = 0: no logit above -inf
    if (sums.s == 0.f) return -INFINITY;
    if (fabsf(x) >= 1e30f) return (x - sums.m) * a.beta - log2_s * kLn2;
    const float p = (above(x, sums.m, r, b2) - log2_s) * kLn2;
    return p > 0.f ? 0.f : p;  // (rounding)
  };
  if (lane == 0) {
    if (a.logprob) {
      const int token = a.tokens[t];
      a.logprob[t] = token >= 0 && token < a.V ? log_p(logit) : -INFINITY;
    }
    if (a.entropy) {
      const float h = sums.s == 0.f ? 0.f : (log2_s - sums.q / sums.s) * kLn2;
      a.entropy[t] = h < 0.f ? 0.f : h;
    }
    if (a.lse) a.lse[t] = sums.s == 0.f ? -INFINITY : fmaf(sums.m, a.beta, (log2_s - Sums::rest(sums.m, b2)) * kLn2);
  }
  if (!a.k) return;
  float v = value_of(list);
  int at = index_of(list);
  // fewer than k logits above -inf: the first of those that are -inf
  int found = (int)__popcll(__ballot(at >= 0));
  if (found < a.k) {
    for (int x0 = 0; x0 < a.V && found < a.k; x0 += 64) {
      const int x = x0 + lane;
      const uint64_t there = __ballot(x < a.V && value_at<TYPE>(row, min(x, a.V - 1)) == -INFINITY);
      const int n = (int)__popcll(there);
      if (lane >= found && lane < found + n) {
        uint64_t rest = there;  // its (lane - found)-th
        for (int i = found; i < lane; i++) rest &= rest - 1;
        at = x0 + __builtin_ctzll(rest);
      }
      found += n;
    }
  }
  if (lane < a.k) {
    a.top[(int64_t)t * a.k + lane] = at;
    a.top_logprob[(int64_t)t * a.k + lane] = at < 0 ? NAN : log_p(v);  // (the others are NaN)
  }
}

template <int TYPE, bool TOP>
__global__ __launch_bounds__(kThreads, 8) void token_logprobs_kernel(LogprobArgs a) {
  __shared__ Sums sums[kWaves];
  __shared__ Entry lists[TOP ? kWaves : 1][128];
  constexpr int RUN = kRun;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x / a.parts, part = blockIdx.x - t * a.parts;
  const char *row = (const char *)a.logits + t * a.stride * (16 / kPer<TYPE>);
  // runs begin at a multiple of 16 bytes
  const int lead = (int)((uintptr_t)row % 16) / (16 / kPer<TYPE>);
  const int runs = (a.V + lead + RUN - 1) / RUN;
  const int lo = (int)((int64_t)runs * part / a.parts), hi = (int)((int64_t)runs * (part + 1) / a.parts);
  const float b2 = a.beta * kLog2e, logit = a.parts == 1 ? logit_of<TYPE>(a, t) : 0.f;
  Wave<TYPE, TOP> w;
  w.sums = Sums{kLowest, 0.f, 0.f};
  w.list = kNone;
  w.last = -INFINITY;
  w.waiting = 0;
  uint4 next[kLoads<TYPE>];
  int x = lo + wave;
  if (x < hi) load<TYPE>(row, a.V, x * RUN - lead, lane, next);
  for (; x < hi; x += kWaves) {
    uint4 now[kLoads<TYPE>];
#pragma unroll
    for (int i = 0; i < kLoads<TYPE>; i++) now[i] = next[i];
    if (x + kWaves < hi) load<TYPE>(row, a.V, (x + kWaves) * RUN - lead, lane, next);
    w.run(now, x * RUN - lead, b2, a.k, lane, lists[TOP ? wave : 0]);
  }
  w.sums.join_lanes(b2);
  if (lane == 0) sums[wave] = w.sums;
  if (TOP) {
    w.take(lists[wave], lane);
    lists[wave][lane] = w.list;
  }
  __syncthreads();
  if (wave) return;
  w.sums = sums[lane % kWaves];
  w.sums.template join_lanes<kWaves>(b2);
  if (TOP) {
#pragma unroll
    for (int i = 1; i < kWaves; i++) w.list = joined(w.list, lists[i][lane], lane);
  }
  if (a.parts == 1) return finish<TYPE>(a, t, logit, w.sums, w.list, lane);
  float *out = a.part + (int64_t)blockIdx.x * (4 + 2 * a.k);
  if (lane == 0) {
    out[0] = w.sums.m;
    out[1] = w.sums.s;
    out[2] = w.sums.q;
  }
  if (TOP && lane < a.k) ((Entry *)(out + 4))[lane] = w.list;
}

// Joins a row's parts: their lists' entries go to the lanes of all waves, each
// wave sorts its 64, and the waves' lists join in pairs.
template <int TYPE>
__global__ __launch_bounds__(64 * kJoinWaves) void join_logprobs_kernel(LogprobArgs a) {
  __shared__ Entry lists[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.x;
  const float b2 = a.beta * kLog2e, logit = logit_of<TYPE>(a, t);
  const size_t words = 4 + 2 * a.k;
  const float *in = a.part + (size_t)t * a.parts * words;
  const int entries = a.parts * a.k, used = min(kJoinWaves, (entries + 63) / 64);
  Entry list = kNone;
  for (int x0 = 64 * wave; x0 < entries; x0 += 64 * kJoinWaves) {
    const int x = x0 + lane, p = x / max(a.k, 1), j = x - p * a.k;
    const Entry o = sorted(x < entries ? ((const Entry *)(in + p * words + 4))[j] : kNone, lane);
    list = x0 < 64 * kJoinWaves ? o : joined(list, o, lane);
  }
  for (int d = 1; d < used; d *= 2) {
    if ((wave & (2 * d - 1)) == d) lists[wave][lane] = list;
    __syncthreads();
    if (!(wave & (2 * d - 1)) && wave + d < used) list = joined(list, lists[wave + d][lane], lane);
  }
  if (wave) return;
  Sums sums = {kLowest, 0.f, 0.f};
  for (int p = lane; p < a.parts; p += 64) sums.join(Sums{in[p * words], in[p * words + 1], in[p * words + 2]}, b2);
  sums.join_lanes(b2);
  finish<TYPE>(a, t, logit, sums, list, lane);
}

template <int TYPE>
hipError_t launch(const LogprobArgs &a, hipStream_t s) {
  const unsigned grid = (unsigned)a.T * a.parts;
  if (a.k) token_logprobs_kernel<TYPE, true><<<grid, kThreads, 0, s>>>(a);
  else token_logprobs_kernel<TYPE, false><<<grid, kThreads, 0, s>>>(a);
  if (a.parts > 1) {
    if (const hipError_t e = hipGetLastError()) return e;
    join_logprobs_kernel<TYPE><<<a.T, 64 * kJoinWaves, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

// Parts of a row: so many that four workgroups are there for each CU, and each
// wave of a part has a run. Every wave has a list of its own to begin and to
// join, so that more of them cost more than they hide: 1000 rows of 150001 fp32
// logits with 20 alternatives take 97 us in one part (four to a CU), 104 in two,
// 110 in four; one row of 131072, for which only latency counts, 11.5 us in 32
// parts, 11.9 in 16 and 13.5 in 8 (with the calls' time on the host).
static int most_parts(int V) { return std::max(1, V / (kWaves * kRun)); }
static int all_parts() { return 4 * num_cus(); }
int logprob_parts(int T, int V) { return std::max(1, std::min(most_parts(V), all_parts() / std::max(T, 1))); }

// Of several parts to a row no more than all_parts() are there, whatever T is:
// as many as so many rows, or fewer, can have.
size_t logprob_workspace_parts(int T, int V) {
  return most_parts(V) == 1 ? 0 : std::min((size_t)T * most_parts(V), (size_t)all_parts());
}

hipError_t launch_token_logprobs(const LogprobArgs &a, hipStream_t s) {
  switch (a.dtype) {
    case K3_BF16: return launch<K3_BF16>(a, s);
    case K3_F16: return launch<K3_F16>(a, s);
    default: return launch<K3_F32>(a, s);
  }
}

}  // namespace k3
