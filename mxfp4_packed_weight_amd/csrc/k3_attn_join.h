// Joins the tiles that were split: workgroup b's is the tile that begins in
// its stretch of the line and goes on in the next ones. A wave joins one row
// at a time, four values per lane, as many parts side by side as lanes allow
// and eight of those in flight: maxima, sums and values of a step's parts are
// loaded together, so a row costs one memory latency per step (the parts are
// few and come from other dies' memory; latency is all that this launch has).
#pragma once

#include <type_traits>

#include "k3_attn.h"

namespace k3 {

constexpr int kJoinWaves = 4;

template <bool BF, int D>
__global__ __launch_bounds__(64 * kJoinWaves) void attn_join_kernel(AttnArgs a, int B) {
  __shared__ int lists[kJoinWaves][kMaxWorkgroups + 1];
  const int b = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const JoinJob *jobs = join_jobs<D>(a, B);
  const JoinJob job = jobs[b];
  if ((int)blockIdx.y * kJoinWaves + wave >= job.rows) return;
  int *slots = lists[wave], n = 0;
  for (int x0 = b; x0 <= job.last; x0 += 64) {
    const int x = x0 + lane;
    const int slot = x > job.last ? -1 : x == b ? job.tail_slot : jobs[x].head_slot;
    const uint64_t there = __ballot(slot >= 0);
    if (slot >= 0) slots[n + __popcll(there & ((1ull << lane) - 1))] = slot;
    n += __popcll(there);
  }
  wave_sync();
  if (n == 0) return;  // one workgroup had all of its blocks
  constexpr int LPR = D / 4, SIDE = 64 / LPR;
  const int sub = lane / LPR, d = lane % LPR * 4;
  for (int r = blockIdx.y * kJoinWaves + wave; r < job.rows; r += gridDim.y * kJoinWaves) {
    float ref = -INFINITY, sum = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    auto weight = [&](float m, float top) { return m == top ? 1.f : exp2_hw(m - top); };
    auto join = [&](auto ahead, int x0) {
      constexpr int kAhead = decltype(ahead)::value;
      f32x4 p[kAhead];
      float m[kAhead], s[kAhead], top = ref;
#pragma unroll
      for (int i = 0; i < kAhead; i++) {
        const int x = x0 + i * SIDE + sub, slot = slots[min(x, n - 1)];
        const float *ml = part_ml<D>(a, B, slot);
        m[i] = ml[r];
        s[i] = ml[a.part_rows + r];
        p[i] = *(const f32x4 *)(part_o<D>(a, slot, r) + d);
      }
#pragma unroll
      for (int i = 0; i < kAhead; i++)
        if (x0 + i * SIDE + sub < n) top = fmaxf(top, m[i]);
      const float keep = weight(ref, top);
      ref = top;
      sum *= keep;
      o *= keep;
#pragma unroll
      for (int i = 0; i < kAhead; i++)
        if (x0 + i * SIDE + sub < n) {
          const float f = weight(m[i], ref);
          sum = fmaf(s[i], f, sum);
          o += p[i] * f;
        }
    };
    int x0 = 0;
    for (; x0 + 2 * SIDE < n; x0 += 8 * SIDE) join(std::integral_constant<int, 8>{}, x0);
    for (; x0 < n; x0 += SIDE) join(std::integral_constant<int, 1>{}, x0);
#pragma unroll
    for (int k = LPR; k < 64; k *= 2) {
      const float m = __shfl_xor(ref, k), top = fmaxf(ref, m);
      const float mine = weight(ref, top), other = weight(m, top);
      ref = top;
      sum = sum * mine + __shfl_xor(sum, k) * other;
#pragma unroll
      for (int i = 0; i < 4; i++) o[i] = o[i] * mine + __shfl_xor(o[i], k) * other;
    }
    if (sub) continue;
    const int row = job.row0 + r, i = row / a.G, hq = job.h * a.G + row - i * a.G;
    const size_t tok = job.t0 + i;
    const float f = sum == 0.f ? 0.f : (a.c.v_scale ? a.c.v_scale[job.h] : 1.f) / sum;
    *(u32x2 *)(a.out + tok * a.out_stride + hq * D + d) =
        u32x2{pack2<BF>(o[0] * f, o[1] * f), pack2<BF>(o[2] * f, o[3] * f)};
    if (a.lse && lane == 0) a.lse[tok * a.Hq + hq] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
  }
}

}  // namespace k3
