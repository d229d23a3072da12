// The residual's addition and the root-mean-square norm, in 16 bits and in e4m3
// with scales.
//
//   s = x + residual,  y = s r w,  r = rsqrt(mean s^2 + eps)
//   scale = max |y| / 448 over a group,  code = e4m3(y / scale)
// A workgroup takes a row, and each thread keeps eight values of one or two
// stretches of it in registers: a row is read once. The largest |y| of a group
// is r times the largest |s w|, so that the row's sum of squares and a scale per
// row need one exchange between the waves, and a group of up to 512 values is
// in neighbouring lanes of a wave. The sum goes into the norm unrounded. Rows
// whose squares leave fp32's range are summed once more, scaled; s stays in registers
// for that (reading the inputs again instead has to hold back the sum, which may go
// over one of them: 4096 rows of 16384 88 -> 101 us).
//
// Bytes bound it: 16384 rows of 7168 with all three outputs, 1.06 GB: 180 us, 5.9
// TB/s (a copy: 5.1); 2048 rows into e4m3 with scales of 128 values, 103 MB: 19 us
// with warm inputs, 22 without. One row takes 2.4 us, and its call on the
// host three times that.
#include "k3_lanes.h"
#include "k3_rows.h"
#include "k3_step.h"

namespace k3 {

namespace {

constexpr int kNormThreads = 1024, kNormWaves = kNormThreads / 64;

// Eight values' products with their weights.
template <bool BF>
__device__ __forceinline__ void weighted(const float *s, const uint4 &weights, float *out) {
  float w[8];
  unpack8<BF>(weights, w);
#pragma unroll
  for (int j = 0; j < 8; j++) out[j] = s[j] * w[j];
}
__device__ __forceinline__ float largest_of(const float *x) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; j++) top = fmaxf(fabsf(x[j]), top);
  return top;
}

template <bool BF, bool QUANT, int VEC>
__global__ __launch_bounds__(kNormThreads) void add_rms_norm_kernel(NormArgs a) {
  __shared__ float sums[kNormWaves], tops[kNormWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t t = blockIdx.x;
  const int vectors = a.hidden / 8;
  float h[VEC][8], hw[VEC][8];
  uint4 xs[VEC], rs[VEC], ws[VEC];
#pragma unroll
  for (int i = 0; i < VEC; i++) {
    const int v = i * blockDim.x + threadIdx.x;
    xs[i] = rs[i] = ws[i] = uint4{0, 0, 0, 0};
    if (v < vectors) {
      xs[i] = *(const uint4 *)(a.x + t * a.x_stride + 8 * v);
      if (a.residual) rs[i] = *(const uint4 *)(a.residual + t * a.residual_stride + 8 * v);
      ws[i] = *(const uint4 *)(a.w + 8 * v);
    }
  }
  float ss = 0.f, top[VEC];
#pragma unroll
  for (int i = 0; i < VEC; i++) {
    const int v = i * blockDim.x + threadIdx.x;
    float r[8];
    unpack8<BF>(xs[i], h[i]);
    unpack8<BF>(rs[i], r);
#pragma unroll
    for (int j = 0; j < 8; j++) {
      h[i][j] += r[j];
      ss = fmaf(h[i][j], h[i][j], ss);
    }
    weighted<BF>(h[i], ws[i], hw[i]);
    top[i] = QUANT ? largest_of(hw[i]) : 0.f;  // (NaN comes back with r)
    if (a.sum && v < vectors) *(uint4 *)(a.sum + t * a.sum_stride + 8 * v) = pack8<BF>(h[i]);
  }
  const bool per_row = QUANT && a.group == a.hidden;
  float most = 0.f;
  // the row's sum, and its largest if that is wanted, from each thread's
  auto of_row = [&](float &sum) {
    if (per_row) {
      most = 0.f;
#pragma unroll
      for (int i = 0; i < VEC; i++) most = fmaxf(top[i], most);
    }
    halving<32>([&](auto d) {
      constexpr int M = decltype(d)::value;
      sum += lane_xor<M>(sum);
      if (QUANT) most = fmaxf(most, lane_xor<M>(most));
    });
    if (lane == 0) {
      sums[wave] = sum;
      tops[wave] = most;
    }
    __syncthreads();
    sum = sums[0];
    most = tops[0];
    for (int i = 1; i < waves; i++) {
      sum += sums[i];
      most = fmaxf(most, tops[i]);
    }
  };
  of_row(ss);
  const float mean = ss / (float)a.hidden + a.eps;
  float r = rsqrtf(mean);
  // The squares have left fp32's range where the rows may not have (fp16's cannot):
  // again, of rows brought into its middle by a power of two (every thread has
  // the same mean). A mean past the range makes r 0.
  constexpr uint32_t kSmall = 0x0d800000u, kInf = 0x7f800000u;  // 2^-100, infinity
  const uint32_t bits = __builtin_amdgcn_readfirstlane(__builtin_bit_cast(uint32_t, mean));
  if (BF && __builtin_expect(bits < kSmall || bits == kInf, 0)) {
    const bool large = !(mean < INFINITY);
    const float power = large ? 0x1p-80f : 0x1p80f;
    float scaled = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; i++)
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float x = h[i][j] * power;
        scaled = fmaf(x, x, scaled);
      }
    __syncthreads();  // (the sums were read)
    of_row(scaled);
    scaled /= (float)a.hidden;
    const bool past = large && !(scaled < 0x1p-32f), zero = !large && scaled + a.eps == 0.f;
    const float factor = rsqrtf(scaled + a.eps * power * power);
    if (!zero) {  // (else 0 times infinity, as it is)
      r = past ? 0.f : 1.f;
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        const int v = i * blockDim.x + threadIdx.x;
        uint4 w = uint4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};  // (ones: 0 times s is 0 or NaN)
        if (!past && v < vectors) w = *(const uint4 *)(a.w + 8 * v);
        // (large: the power belongs to the factor, which it does not take out of range; small: to the value)
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (!past) h[i][j] = large ? h[i][j] * (factor * power) : h[i][j] * power * factor;
        weighted<BF>(h[i], w, hw[i]);
        top[i] = QUANT ? largest_of(hw[i]) : 0.f;
      }
      if (per_row) {
        float none = 0.f;
        __syncthreads();
        of_row(none);
      }
    }
  }
  // a group's lanes, and their logarithm (divisions by them took 0.7 us of 21.7, 2048
  // rows into e4m3, whose bound is the vector unit as much as the bytes)
  const int lanes = per_row ? 64 : a.group / 8, shift = per_row ? 31 : 31 - __builtin_clz(lanes | 1);
#pragma unroll
  for (int i = 0; i < VEC; i++) {
    const int v = i * blockDim.x + threadIdx.x;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j++) y[j] = hw[i][j] * r;
    if (a.y && v < vectors) *(uint4 *)(a.y + t * a.y_stride + 8 * v) = pack8<BF>(y);
    if (QUANT) {
      float largest = most;
      if (!per_row) {  // over the group's lanes
        largest = fmaxf(top[i], lane_xor<1>(top[i]));
        largest = fmaxf(largest, lane_xor<2>(largest));
        if (lanes >= 8) largest = fmaxf(largest, lane_xor<4>(largest));
        if (lanes >= 16) largest = fmaxf(largest, lane_xor<8>(largest));
        if (lanes >= 32) largest = fmaxf(largest, lane_xor<16>(largest));
        if (lanes >= 64) largest = fmaxf(largest, lane_xor<32>(largest));
      }
      if (v >= vectors) continue;
      float scale = largest * r * (1.f / 448.f);
      if (scale < 0x1p-126f) scale = 0.f;  // (not for NaN)
      // (at most 448 and four roundings, which is 448 in e4m3; r / scale may be infinite)
      const float up = scale == 0.f ? 0.f : 1.f / scale;
#pragma unroll
      for (int j = 0; j < 8; j++) y[j] *= up;
      *(uint2 *)(a.y8 + t * a.y8_stride + 8 * v) = to_e4m3(y);
      if ((v & ((1u << shift) - 1)) == 0) a.scales[t * (per_row ? 1 : vectors >> shift) + (v >> shift)] = scale;
    }
  }
}

template <bool BF, bool QUANT>
hipError_t by_vectors(const NormArgs &a, hipStream_t s) {
  const int vectors = a.hidden / 8;
  auto threads = [&](int vec) { return ((vectors + vec - 1) / vec + 63) / 64 * 64; };
  // Threads of one vector where each row has a CU to itself (one row of 7168 2.38 us,
  // of two 2.57; 255 rows 3.67 and 3.80), else of two: 2048 rows of 7168 into e4m3
  // 24.1 us (cold), of one 26.5, of four 25.7, of eight 39.6.
  const int vec = vectors <= kNormThreads && a.T < num_cus() ? 1 : 2;
  if (vec == 1) add_rms_norm_kernel<BF, QUANT, 1><<<a.T, threads(1), 0, s>>>(a);
  else add_rms_norm_kernel<BF, QUANT, 2><<<a.T, threads(2), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs &a, hipStream_t s) {
  if (a.dtype == K3_BF16) return a.y8 ? by_vectors<true, true>(a, s) : by_vectors<true, false>(a, s);
  return a.y8 ? by_vectors<false, true>(a, s) : by_vectors<false, false>(a, s);
}

}  // namespace k3
