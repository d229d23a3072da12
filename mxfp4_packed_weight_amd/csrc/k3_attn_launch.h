// Which attention kernel a call takes, and its launches.
#pragma once

#include "k3_attn_stream.h"

namespace k3 {

template <bool BF, bool F8, int D, int QT>
hipError_t launch_stream(const AttnArgs &a, hipStream_t s) {
  constexpr int RT = 16 * QT;
  const int B = attn_workgroups();
  const size_t pre = (a.R + 1) * sizeof(long long);
  attn_stream_kernel<BF, F8, D, QT><<<B, kStreamThreads, pre, s>>>(a);
  if (const hipError_t e = hipGetLastError()) return e;
  attn_join_kernel<BF, D, RT, kStreamKeys><<<dim3(B, RT / 4), 256, pre, s>>>(a, B);
  return hipGetLastError();
}

template <bool BF, bool F8, int D>
hipError_t launch_attn(const AttnArgs &a, hipStream_t s) {
  switch (attn_tile_rows(a.T, a.G, a.R, D)) {
    case 16: return launch_stream<BF, F8, D, 1>(a, s);
    case 32: return launch_stream<BF, F8, D, 2>(a, s);
    default:
      if constexpr (D < 256) return launch_stream<BF, F8, D, 4>(a, s);
      return hipErrorInvalidValue;
  }
}

template <bool BF, bool F8>
hipError_t attn_by_dim(const AttnArgs &a, hipStream_t s) {
  switch (a.c.head_dim) {
    case 64: return launch_attn<BF, F8, 64>(a, s);
    case 128: return launch_attn<BF, F8, 128>(a, s);
    default: return launch_attn<BF, F8, 256>(a, s);
  }
}

}  // namespace k3
