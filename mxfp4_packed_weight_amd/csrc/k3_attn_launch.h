// Which attention kernel a call takes, and its launches.
#pragma once

#include "k3_attn_join.h"
#include "k3_attn_stream.h"
#include "k3_attn_tile.h"

namespace k3 {

template <bool BF, int D>
hipError_t launch_join(const AttnArgs &a, int B, hipStream_t s) {
  if (const hipError_t e = hipGetLastError()) return e;
  attn_join_kernel<BF, D><<<join_workgroups(a, B), 64 * kJoinWaves, 0, s>>>(a, B);
  return hipGetLastError();
}

template <bool BF, bool F8, int D, int QT>
hipError_t launch_stream(const AttnArgs &a, hipStream_t s) {
  const int B = attn_workgroups(16 * QT, D);
  attn_stream_kernel<BF, F8, D, QT><<<B, kStreamThreads, 0, s>>>(a);
  return launch_join<BF, D>(a, B, s);
}

template <bool BF, bool F8, int D>
hipError_t launch_tile(const AttnArgs &a, hipStream_t s) {
  const int B = attn_workgroups(32 * kAttnWaves<D>, D);
  attn_tile_kernel<BF, F8, D><<<B, kAttnThreads<D>, 0, s>>>(a);
  return launch_join<BF, D>(a, B, s);
}

template <bool BF, bool F8, int D>
hipError_t launch_attn(const AttnArgs &a, hipStream_t s) {
  switch (attn_tile_rows(a.T, a.G, a.R, D)) {
    case 16: return launch_stream<BF, F8, D, 1>(a, s);
    case 32:
      if constexpr (D < 256) return launch_stream<BF, F8, D, 2>(a, s);
      return hipErrorInvalidValue;
    default: return launch_tile<BF, F8, D>(a, s);
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
