// Log probabilities of given tokens, entropy, and the largest logits of rows.
//
//   z = beta x,  lse = log sum exp z,  log p = z - lse,
//   entropy = log S - Q / S,  S = sum e^d, Q = sum e^d d, d = z - beta m,
// for a reference m that is at least near the largest of what was read so far:
// one pass, S and Q are scaled when m rises. Differences are taken before the
// factor beta, so that logits of the type's lowest value still differ by 0 from
// one another. In e^d d an x of
// -inf counts as the lowest number, times 0.
//
// A row's logits go to the waves in runs of 64 lanes x 2 loads of 16 bytes. Each
// wave keeps the k <= 64 largest of its logits sorted in its lanes, one a lane:
// only a logit above the k-th is looked at, from the lowest lane on, which
// leaves equal ones in the order of their indices. The first run's threshold is
// the k-th largest of the lanes' own maxima. Lists join by comparing one with
// another turned round, which leaves the largest 64 of both, and six steps of
// sorting.
#include <math.h>

#include <algorithm>

#include "k3_rows.h"
#include "k3_step.h"

namespace k3 {

namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves, kJoinWaves = 8;
constexpr int kLoads = 2;  // of a lane in a run
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.4028234663852886e38f;

template <int TYPE>
constexpr int kPer = TYPE == K3_F32 ? 4 : 8;  // values of 16 bytes
template <int TYPE>
constexpr int kRun = 64 * kLoads * kPer<TYPE>;

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

struct Sums {
  float m, s, q;
  // what is known of values below a higher reference, seen from it (x log2e beta = b2)
  __device__ __forceinline__ void raise(float top, float b2) {
    const float f = m == top ? 1.f : exp2f((m - top) * b2);
    q = f == 0.f ? 0.f : f * (q - (top - m) * s);
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
};

// ---- lists of the largest -------------------------------------------------------

// Lane j has the j-th largest, or (-inf, INT_MAX).
struct List {
  float v;
  int at;
};
// Greater values first, of equal ones the lower index.
__device__ __forceinline__ bool before(const List &x, const List &y) {
  return x.v > y.v || (x.v == y.v && x.at < y.at);
}
__device__ __forceinline__ float of_lane(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}
// The largest 64 of both.
__device__ __forceinline__ List joined(List x, const List &y, int lane) {
  List o = {__shfl(y.v, 63 - lane), __shfl(y.at, 63 - lane)};
  if (before(o, x)) x = o;
#pragma unroll
  for (int d = 32; d; d /= 2) {
    o = List{__shfl_xor(x.v, d), __shfl_xor(x.at, d)};
    if (before(o, x) == !(lane & d)) x = o;
  }
  return x;
}
// A list of any 64 entries.
__device__ __forceinline__ List sorted(List x, int lane) {
#pragma unroll
  for (int n = 2; n <= 64; n *= 2)
#pragma unroll
    for (int d = n / 2; d; d /= 2) {
      const List o = {__shfl_xor(x.v, d), __shfl_xor(x.at, d)};
      if (before(o, x) == (!(lane & d) == !(lane & n))) x = o;
    }
  return x;
}
// Puts a value in (all lanes the same; larger than the list's last).
__device__ __forceinline__ void insert(List &x, float v, int at, int lane) {
  const int place = __popcll(__ballot(x.v >= v));
  const float pv = __shfl_up(x.v, 1);
  const int pat = __shfl_up(x.at, 1);
  if (lane > place) x = List{pv, pat};
  if (lane == place) x = List{v, at};
}
// Rising integers for rising floats, and back.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __builtin_bit_cast(float, u & 0x80000000u ? u & 0x7fffffffu : ~u);
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
  for (int i = 0; i < kLoads; i++) {
    const int at = first + (i * 64 + lane) * PER;
    if (at >= 0 && at <= V - PER) {
      out[i] = *(const uint4 *)(row + (int64_t)at * ES);
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
  List list;
  float last;  // what a logit must be above to be looked at

  __device__ __forceinline__ void run(const uint4 *in, int first, float b2, int k, int lane, bool begin) {
    constexpr int PER = kPer<TYPE>;
    float x[kLoads][PER], most[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      unpack<TYPE>(in[i], x[i]);
      most[i] = x[i][0];
#pragma unroll
      for (int j = 1; j < PER; j++) most[i] = fmaxf(most[i], x[i][j]);
    }
    float top = most[0];
#pragma unroll
    for (int i = 1; i < kLoads; i++) top = fmaxf(top, most[i]);
    if (__ballot((top - sums.m) * b2 > 1.f)) sums.raise(fmaxf(sums.m, top), b2);
#pragma unroll
    for (int i = 0; i < kLoads; i++)
#pragma unroll
      for (int j = 0; j < PER; j++) {
        const float d = x[i][j] - sums.m, e = __builtin_amdgcn_exp2f(d * b2);
        sums.s += e;
        sums.q = fmaf(e, fmaxf(d, kLowest), sums.q);  // (0 times -inf is none)
      }
    if (!TOP) return;
    if (begin) last = below_kth(top == top ? top : -INFINITY, k);
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      uint64_t lanes = __ballot(most[i] > last);
      while (lanes) {
        const int l = __builtin_ctzll(lanes);
#pragma unroll
        for (int j = 0; j < PER; j++) {
          const float v = of_lane(x[i][j], l) + 0.f;  // (no -0)
          if (v > last) {
            insert(list, v, first + (i * 64 + l) * PER + j, lane);
            last = fmaxf(last, of_lane(list.v, k - 1));
          }
        }
        lanes = __ballot(most[i] > last) & ~((2ull << l) - 1);
      }
    }
  }
};

template <int TYPE>
__device__ void finish(const LogprobArgs &a, int t, Sums sums, List list, int lane) {
  const char *row = (const char *)a.logits + t * a.stride * (16 / kPer<TYPE>);
  const float log2_s = log2f(sums.s);
  auto log_p = [&](float x) {  // S = 0: no logit above -inf
    return sums.s == 0.f ? -INFINITY : (x - sums.m) * a.beta - log2_s * kLn2;
  };
  if (lane == 0) {
    if (a.logprob) {
      const int token = a.tokens[t];
      a.logprob[t] = token >= 0 && token < a.V ? log_p(value_at<TYPE>(row, token)) : -INFINITY;
    }
    if (a.entropy) {
      const float h = sums.s == 0.f ? 0.f : log2_s * kLn2 - a.beta * (sums.q / sums.s);
      a.entropy[t] = h < 0.f ? 0.f : h;
    }
    if (a.lse) a.lse[t] = sums.s == 0.f ? -INFINITY : fmaf(sums.m, a.beta, log2_s * kLn2);
  }
  if (!a.k) return;
  // fewer than k logits above -inf: the first of those that are -inf
  int found = __popcll(__ballot(list.at != 0x7fffffff));
  if (found < a.k) {
    for (int x0 = 0; x0 < a.V && found < a.k; x0 += 64) {
      const int x = x0 + lane;
      const uint64_t there = __ballot(x < a.V && value_at<TYPE>(row, min(x, a.V - 1)) == -INFINITY);
      const int n = __popcll(there);
      if (lane >= found && lane < found + n) {
        uint64_t rest = there;  // its (lane - found)-th
        for (int i = found; i < lane; i++) rest &= rest - 1;
        list.at = x0 + __builtin_ctzll(rest);
      }
      found += n;
    }
  }
  if (lane < a.k) {
    const bool none = list.at == 0x7fffffff;  // the others are NaN
    a.top[(int64_t)t * a.k + lane] = none ? -1 : list.at;
    a.top_logprob[(int64_t)t * a.k + lane] = none ? NAN : log_p(list.v);
  }
}

template <int TYPE, bool TOP>
__global__ __launch_bounds__(kThreads) void token_logprobs_kernel(LogprobArgs a) {
  __shared__ Sums sums[kWaves];
  __shared__ List lists[kWaves][64];
  constexpr int RUN = kRun<TYPE>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x / a.parts, part = blockIdx.x - t * a.parts;
  const char *row = (const char *)a.logits + t * a.stride * (16 / kPer<TYPE>);
  // runs begin at a multiple of 16 bytes
  const int lead = (int)((uintptr_t)row % 16) / (16 / kPer<TYPE>);
  const int runs = (a.V + lead + RUN - 1) / RUN;
  const int lo = (int)((int64_t)runs * part / a.parts), hi = (int)((int64_t)runs * (part + 1) / a.parts);
  const float b2 = a.beta * kLog2e;
  Wave<TYPE, TOP> w;
  w.sums = Sums{kLowest, 0.f, 0.f};
  w.list = List{-INFINITY, 0x7fffffff};
  w.last = -INFINITY;
  uint4 next[kLoads];
  int x = lo + wave;
  if (x < hi) load<TYPE>(row, a.V, x * RUN - lead, lane, next);
  for (; x < hi; x += kWaves) {
    uint4 now[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; i++) now[i] = next[i];
    if (x + kWaves < hi) load<TYPE>(row, a.V, (x + kWaves) * RUN - lead, lane, next);
    w.run(now, x * RUN - lead, b2, a.k, lane, x == lo + wave);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2)
    w.sums.join(Sums{__shfl_xor(w.sums.m, d), __shfl_xor(w.sums.s, d), __shfl_xor(w.sums.q, d)}, b2);
  if (lane == 0) sums[wave] = w.sums;
  if (TOP) lists[wave][lane] = w.list;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int i = 1; i < kWaves; i++) {
    w.sums.join(sums[i], b2);
    if (TOP) w.list = joined(w.list, lists[i][lane], lane);
  }
  if (a.parts == 1) return finish<TYPE>(a, t, w.sums, w.list, lane);
  float *out = a.part + (int64_t)blockIdx.x * (4 + 2 * a.k);
  if (lane == 0) {
    out[0] = w.sums.m;
    out[1] = w.sums.s;
    out[2] = w.sums.q;
  }
  if (TOP && lane < a.k) {
    out[4 + lane] = w.list.v;
    ((int *)out)[4 + a.k + lane] = w.list.at;
  }
}

// Joins a row's parts: their lists' entries go to the lanes of all waves, each
// wave sorts its 64, and the waves' lists join in pairs.
template <int TYPE>
__global__ __launch_bounds__(64 * kJoinWaves) void join_logprobs_kernel(LogprobArgs a) {
  __shared__ List lists[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.x;
  const float b2 = a.beta * kLog2e;
  const size_t words = 4 + 2 * a.k;
  const float *in = a.part + (size_t)t * a.parts * words;
  const int entries = a.parts * a.k, used = min(kJoinWaves, (entries + 63) / 64);
  List list = {-INFINITY, 0x7fffffff};
  for (int x0 = 64 * wave; x0 < entries; x0 += 64 * kJoinWaves) {
    const int x = x0 + lane, p = x / max(a.k, 1), j = x - p * a.k;
    List o = {-INFINITY, 0x7fffffff};
    if (x < entries) o = List{in[p * words + 4 + j], ((const int *)in)[p * words + 4 + a.k + j]};
    o = sorted(o, lane);
    list = x0 < 64 * kJoinWaves ? o : joined(list, o, lane);
  }
  for (int d = 1; d < used; d *= 2) {
    if (wave & d) lists[wave][lane] = list;
    __syncthreads();
    if (!(wave & (2 * d - 1)) && wave + d < used) list = joined(list, lists[wave + d][lane], lane);
  }
  if (wave) return;
  Sums sums = {kLowest, 0.f, 0.f};
  for (int p = lane; p < a.parts; p += 64) sums.join(Sums{in[p * words], in[p * words + 1], in[p * words + 2]}, b2);
#pragma unroll
  for (int d = 1; d < 64; d *= 2)
    sums.join(Sums{__shfl_xor(sums.m, d), __shfl_xor(sums.s, d), __shfl_xor(sums.q, d)}, b2);
  finish<TYPE>(a, t, sums, list, lane);
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

// Parts of a row: so many that the card is full, and each wave of a part has a
// run of 16-bit logits.
int logprob_parts(int T, int V) {
  const int most = std::max(1, V / (kWaves * kRun<K3_BF16>));
  return std::max(1, std::min(most, 8 * num_cus() / std::max(T, 1)));
}

hipError_t launch_token_logprobs(const LogprobArgs &a, hipStream_t s) {
  switch (a.dtype) {
    case K3_BF16: return launch<K3_BF16>(a, s);
    case K3_F16: return launch<K3_F16>(a, s);
    default: return launch<K3_F32>(a, s);
  }
}

}  // namespace k3
