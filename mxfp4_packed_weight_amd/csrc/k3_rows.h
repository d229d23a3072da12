// Rows of 16-bit values, eight to a lane.
#pragma once

#include "k3_internal.h"

namespace k3 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

template <bool BF>
__device__ __forceinline__ void unpack8(const uint4 &p, float *f) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if (BF) {
      f[2 * i] = __builtin_bit_cast(float, w[i] << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
    } else {
      const f16x2 h = __builtin_bit_cast(f16x2, w[i]);
      f[2 * i] = (float)h[0];
      f[2 * i + 1] = (float)h[1];
    }
  }
}

template <bool BF>
__device__ __forceinline__ uint4 pack8(const float *f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const f32x2 v = {f[2 * i], f[2 * i + 1]};
    if (BF) w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    else w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
  }
  return uint4{w[0], w[1], w[2], w[3]};
}

// Eight values in e4m3, round to nearest even (none is past 448; NaN stays NaN).
__device__ __forceinline__ uint2 to_e4m3(const float *y) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
  return uint2{(uint32_t)lo, (uint32_t)hi};
}

}  // namespace k3
