// What the lanes of a wave do among themselves.
#pragma once

#include <type_traits>

#include "k3_internal.h"

namespace k3 {

// Orders a wave's own LDS accesses, which its lanes share (LDS serves a
// wave's accesses in order; this keeps the compiler to that order).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// x of lane l ^ D, without a way through LDS: a few cycles, where __shfl_xor
// takes about a hundred.
template <int D>
__device__ __forceinline__ uint32_t lane_xor(uint32_t x) {
  static_assert(D == 1 || D == 2 || D == 4 || D == 8 || D == 16 || D == 32, "");
  constexpr int kQuad1 = 0xb1, kQuad2 = 0x4e, kQuad3 = 0x1b, kMirror8 = 0x141, kRotate8 = 0x128;
  auto dpp = [](uint32_t v, auto control) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(control)::value, 0xf, 0xf, false);
  };
  if constexpr (D == 1) return dpp(x, std::integral_constant<int, kQuad1>{});
  if constexpr (D == 2) return dpp(x, std::integral_constant<int, kQuad2>{});
  if constexpr (D == 4)  // 7, then 3
    return dpp(dpp(x, std::integral_constant<int, kMirror8>{}), std::integral_constant<int, kQuad3>{});
  if constexpr (D == 8) return dpp(x, std::integral_constant<int, kRotate8>{});
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  // the swap of two copies leaves the lower lanes' values in one, the upper ones' in the other
  const u32x2 s = D == 16 ? __builtin_amdgcn_permlane16_swap(x, x, false, false)
                          : __builtin_amdgcn_permlane32_swap(x, x, false, false);
  const uint32_t lower = s[0], upper = s[1];
  return lane & D ? lower : upper;
}
template <int D>
__device__ __forceinline__ float lane_xor(float x) {
  return __builtin_bit_cast(float, lane_xor<D>(__builtin_bit_cast(uint32_t, x)));
}

// f(std::integral_constant<int, D>) for D = FROM, FROM / 2, ..., 1.
template <int FROM, class F>
__device__ __forceinline__ void halving(F &&f) {
  f(std::integral_constant<int, FROM>{});
  if constexpr (FROM > 1) halving<FROM / 2>(f);
}

}  // namespace k3
