// Query/key norm per head, rotation, and the append to the paged cache.
//
// A wave takes a token's heads in passes: eight values per lane (16 bytes in,
// 16 out), D / 8 lanes per head, 512 / D heads per pass. Which values a lane
// holds never changes, so its cosines and sines, and its norm weights times
// them, stay in registers for all of the token's heads:
//   out_a = r (x_a w_a cos) + r (x_b w_b (-+sin)),  r = rsqrt(mean x^2 + eps),
// and the partner x_b comes from the lane that holds it (or is the neighbour
// value when pairs are adjacent), before the norm, in the type it has.
// Angles are fp64: position * inv_freq reaches 1e5 turns of which only the
// fraction counts; reduced to [-pi/4, pi/4] there, then the Taylor series of
// sin and cos to x^11 and x^10 in fp32 (remainders below 2e-10, far under half
// a unit of fp32).
//
// Bytes bound it: each row is read and written once, and the arithmetic
// (about 80 instructions a pass) hides under that. 16384 tokens of 64 query and
// 8 key heads of 128, 671 MB: 142 us, 4.7 TB/s (a copy: 5.0). Few tokens are
// bound by latency: slot and position, then the frequencies (the branch on
// `turns` has each of a lane's four or eight loads waited for by itself), the
// weights and the rows follow one another. 1000 tokens over an e4m3 cache, 19
// MB: 8.4 us, of which 3.9 are the bytes'.
#include "k3_kv.h"
#include "k3_rows.h"

namespace k3 {

namespace {

// x / scale in e4m3, saturated at +-448 (NaN stays NaN), round to nearest even.
__device__ __forceinline__ uint2 pack8_e4m3(const float *f, float scale) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float q = f[i] / scale;
    y[i] = q != q ? q : fminf(fmaxf(q, -448.f), 448.f);
  }
  return to_e4m3(y);
}

__device__ __forceinline__ void sin_cos(double a, float *s, float *c) {
  const double turns = __builtin_rint(a * 0.63661977236758134308);  // 2 / pi
  double x2 = fma(-turns, 1.57079632679489661923, a);
  x2 = fma(-turns, 6.123233995736766e-17, x2);  // pi / 2 past fp64
  const int quad = (int)(long long)turns & 3;
  const float x = (float)x2, y = x * x;
  const float sn = x * fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.f / 39916800.f, 1.f / 362880.f), -1.f / 5040.f),
                                           1.f / 120.f), -1.f / 6.f), 1.f);
  const float cs = fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f),
                                       1.f / 24.f), -0.5f), 1.f);
  const float p = quad & 1 ? cs : sn, q = quad & 1 ? sn : cs;
  *s = quad & 2 ? -p : p;
  *c = (quad + 1) & 2 ? -q : q;
}

// Sum over the LPH lanes of a head.
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int m = 1; m < LPH; m *= 2) v += __shfl_xor(v, m);
  return v;
}

constexpr int kQkWaves = 4;

template <bool BF, bool E4M3, bool INTER, int D>
__global__ __launch_bounds__(kQkWaves * 64) void qk_norm_rope_kernel(QkArgs a, int splits) {
  constexpr int LPH = D / 8, HPP = 64 / LPH;  // lanes per head, heads per pass
  constexpr int kAhead = 4;                   // passes in flight
  const int lane = threadIdx.x & 63;
  const long long unit = (long long)blockIdx.x * kQkWaves + (threadIdx.x >> 6);
  const int t = (int)(unit / splits), part = (int)(unit - (long long)t * splits);
  if (t >= a.T) return;
  const int sub = lane / LPH, d0 = (lane % LPH) * 8;
  const int H = a.c.n_heads, half = a.rot / 2;
  const int q_passes = (a.Hq + HPP - 1) / HPP, k_passes = (H + HPP - 1) / HPP;
  const int passes = q_passes + 2 * k_passes;
  const int lo = (int)((long long)passes * part / splits), hi = (int)((long long)passes * (part + 1) / splits);
  const int slot = a.slots[t];
  const bool kept = slot >= 0 && slot < a.c.n_pages * a.c.page_size;
  const int page = kept ? slot / a.c.page_size : 0, place = kept ? slot - page * a.c.page_size : 0;
  const int64_t cache_row = page * a.c.page_stride + place * a.c.slot_stride + d0;

  // cos and signed sin of this lane's values; lanes past `rot` turn nothing
  const bool turns = d0 < a.rot;
  const int mate = INTER || !turns ? lane : (d0 < half ? lane + half / 8 : lane - half / 8);
  float cs[8], sn[8];
  if (lo < q_passes + k_passes) {
    const double pos = (double)a.positions[t];
#pragma unroll
    for (int j = 0; j < (INTER ? 4 : 8); j++) {
      float s = 0.f, c = 1.f;
      if (turns) {
        const int i = INTER ? d0 / 2 + j : (d0 < half ? d0 + j : d0 - half + j);
        sin_cos(pos * (double)a.inv_freq[i], &s, &c);
      }
      if (INTER) {
        cs[2 * j] = cs[2 * j + 1] = c;
        sn[2 * j] = -s;
        sn[2 * j + 1] = s;
      } else {
        cs[j] = c;
        sn[j] = d0 < half ? -s : s;
      }
    }
  }
  float wc[8], ws[8];  // own weight times cos, partner's times signed sin
  auto weights = [&](const uint16_t *w) {
    float wo[8], wm[8];
    unpack8<BF>(*(const uint4 *)(w + d0), wo);
    const int dm = INTER ? d0 : (mate % LPH) * 8;
    unpack8<BF>(*(const uint4 *)(w + dm), wm);
#pragma unroll
    for (int j = 0; j < 8; j++) {
      wc[j] = wo[j] * cs[j];
      ws[j] = wm[INTER ? j ^ 1 : j] * sn[j];
    }
  };
  auto normed = [&](const uint4 &raw, float *out) {
    float x[8], m[8];
    unpack8<BF>(raw, x);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j++) ss = fmaf(x[j], x[j], ss);
    ss = head_sum<LPH>(ss);
    const float r = rsqrtf(ss * (1.f / D) + a.eps);
    if (!INTER) {
      uint4 other;
      other.x = __shfl(raw.x, mate);
      other.y = __shfl(raw.y, mate);
      other.z = __shfl(raw.z, mate);
      other.w = __shfl(raw.w, mate);
      unpack8<BF>(other, m);
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float y = x[j] * wc[j];
      out[j] = (turns ? fmaf(INTER ? x[j ^ 1] : m[j], ws[j], y) : y) * r;
    }
  };

  // queries
  if (lo < q_passes) {
    weights(a.wq);
    const int end = min(hi, q_passes);
    const uint16_t *in = a.q + t * a.q_stride + d0;
    uint16_t *out = a.q_out + t * a.q_out_stride + d0;
    for (int p0 = lo; p0 < end; p0 += kAhead) {
      uint4 raw[kAhead];
#pragma unroll
      for (int p = 0; p < kAhead; p++) {
        const int h = (p0 + p) * HPP + sub;
        raw[p] = uint4{0, 0, 0, 0};
        if (p0 + p < end && h < a.Hq) raw[p] = *(const uint4 *)(in + h * D);
      }
#pragma unroll
      for (int p = 0; p < kAhead; p++) {
        if (p0 + p >= end) break;
        const int h = (p0 + p) * HPP + sub;
        float y[8];
        normed(raw[p], y);
        if (h < a.Hq) *(uint4 *)(out + h * D) = pack8<BF>(y);
      }
    }
  }
  // keys, then values
  if (hi > q_passes && lo < q_passes + k_passes) weights(a.wk);
  for (int p = max(lo, q_passes); p < hi; p++) {
    const bool is_k = p < q_passes + k_passes;
    const int h = (p - q_passes - (is_k ? 0 : k_passes)) * HPP + sub;
    const bool on = h < H;
    uint4 raw = {0, 0, 0, 0};
    if (on) raw = *(const uint4 *)((is_k ? a.k + t * a.k_stride : a.v + t * a.v_stride) + h * D + d0);
    float y[8];
    if (is_k) normed(raw, y);
    else unpack8<BF>(raw, y);
    if (!on || !kept) continue;
    const int64_t at = cache_row + h * a.c.head_stride;
    if (E4M3) {
      const float *scales = is_k ? a.c.k_scale : a.c.v_scale;
      *(uint2 *)((uint8_t *)(is_k ? a.c.k : a.c.v) + at) = pack8_e4m3(y, scales ? scales[h] : 1.f);
    } else {
      *(uint4 *)((uint16_t *)(is_k ? a.c.k : a.c.v) + at) = is_k ? pack8<BF>(y) : raw;
    }
  }
}

template <bool BF, bool E4M3, bool INTER, int D>
hipError_t launch(const QkArgs &a, hipStream_t s) {
  constexpr int HPP = 512 / D;
  const int passes = (a.Hq + HPP - 1) / HPP + 2 * ((a.c.n_heads + HPP - 1) / HPP);
  // Few tokens: a token's heads go to several waves, each with the angles of
  // its own, until four waves per SIMD are there.
  const int splits = max(1, min(passes, num_cus() * 16 / a.T));
  const long long units = (long long)a.T * splits;
  qk_norm_rope_kernel<BF, E4M3, INTER, D>
      <<<(unsigned)((units + kQkWaves - 1) / kQkWaves), kQkWaves * 64, 0, s>>>(a, splits);
  return hipGetLastError();
}

template <bool BF, bool E4M3, bool INTER>
hipError_t by_dim(const QkArgs &a, hipStream_t s) {
  switch (a.c.head_dim) {
    case 64: return launch<BF, E4M3, INTER, 64>(a, s);
    case 128: return launch<BF, E4M3, INTER, 128>(a, s);
    default: return launch<BF, E4M3, INTER, 256>(a, s);
  }
}

template <bool BF>
hipError_t by_cache(const QkArgs &a, hipStream_t s) {
  if (a.c.dtype == K3_E4M3) return a.interleaved ? by_dim<BF, true, true>(a, s) : by_dim<BF, true, false>(a, s);
  return a.interleaved ? by_dim<BF, false, true>(a, s) : by_dim<BF, false, false>(a, s);
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkArgs &a, hipStream_t s) {
  return a.dtype == K3_BF16 ? by_cache<true>(a, s) : by_cache<false>(a, s);
}

}  // namespace k3
