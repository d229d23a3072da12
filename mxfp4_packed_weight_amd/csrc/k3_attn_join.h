// Joins the tiles that were split: workgroup b's is the tile that begins in
// its stretch of the line and goes on in the next ones. The parts come from
// other dies' memory, and latency is all that this launch has: loads of
// several rows or parts go out together. Tiles in few parts: four values of
// four rows per thread, part by part. Tiles in many (long rows of few
// requests): a wave per row, as many parts side by side as lanes allow and
// up to sixteen of those in flight. One token over 4096 places: 5 us after the
// main launch's 11; 32 trees of up to 64 nodes, 47 MB of parts: 16 us.
#pragma once

#include <algorithm>
#include <type_traits>

#include "k3_attn.h"

namespace k3 {

constexpr int kJoinWaves = 4, kFewParts = 6;

template <bool BF, int D>
__global__ __launch_bounds__(64 * kJoinWaves) void attn_join_kernel(AttnArgs a, int B) {
  __shared__ int lists[kJoinWaves][kMaxWorkgroups + 1], jobs_of[kMaxWorkgroups], found[kJoinWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const JoinJob *jobs = join_jobs<D>(a, B);
  // the jobs that there are, shared out to the workgroups
  int count = 0;
  for (int x0 = 0; x0 < B; x0 += 64 * kJoinWaves) {
    const int x = x0 + threadIdx.x;
    const bool there = x < B && jobs[x].rows > 0;
    const uint64_t all = __ballot(there);
    if (lane == 0) found[wave] = __popcll(all);
    __syncthreads();
    int at = count + __popcll(all & ((1ull << lane) - 1));
    for (int w = 0; w < kJoinWaves; w++) {
      if (w < wave) at += found[w];
      count += found[w];
    }
    if (there) jobs_of[at] = x;
    __syncthreads();
  }
  const int share = blockIdx.x % max(count, 1), chunk = blockIdx.x / max(count, 1);
  const int chunks = ((int)gridDim.x - share + count - 1) / max(count, 1);
  if (count == 0) return;
  const int b = __builtin_amdgcn_readfirstlane(jobs_of[share]);
  const JoinJob job = jobs[b];
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
  const int d = lane % LPR * 4;
  auto weight = [&](float m, float top) { return m == top ? 1.f : exp2_hw(m - top); };
  auto store = [&](int r, float ref, float sum, f32x4 o) {
    const int row = job.row0 + r, i = node_of(a, row), hq = job.h * a.G + row - i * a.G;
    const size_t tok = job.t0 + i;
    const float f = sum == 0.f ? 0.f : (a.c.v_scale ? a.c.v_scale[job.h] : 1.f) / sum;
    *(u32x2 *)(a.out + tok * a.out_stride + hq * D + d) =
        u32x2{pack2<BF>(o[0] * f, o[1] * f), pack2<BF>(o[2] * f, o[3] * f)};
    if (a.lse && d == 0) a.lse[tok * a.Hq + hq] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
  };
  if (n <= kFewParts) {
    constexpr int ROWS = 4, PASS = 64 * kJoinWaves / LPR;  // rows of a thread, rows side by side
    for (int r0 = chunk * ROWS * PASS; r0 < job.rows; r0 += chunks * ROWS * PASS) {
      float ref[ROWS], sum[ROWS];
      f32x4 o[ROWS];
#pragma unroll 2
      for (int x = 0; x < n; x++) {
        const int slot = __builtin_amdgcn_readfirstlane(slots[x]);
        const float *ml = part_ml<D>(a, B, slot), *po = part_o<D>(a, slot, 0) + d;
        float m[ROWS], s[ROWS];
        f32x4 p[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; i++) {
          const int r = min(r0 + i * PASS + (int)threadIdx.x / LPR, job.rows - 1);
          m[i] = ml[r];
          s[i] = ml[a.part_rows + r];
          p[i] = *(const f32x4 *)(po + r * D);
        }
#pragma unroll
        for (int i = 0; i < ROWS; i++) {
          const float top = x ? fmaxf(ref[i], m[i]) : m[i];
          const float mine = x ? weight(ref[i], top) : 0.f, other = weight(m[i], top);
          sum[i] = x ? sum[i] * mine + s[i] * other : s[i];
          o[i] = x ? o[i] * mine + p[i] * other : p[i];
          ref[i] = top;
        }
      }
#pragma unroll
      for (int i = 0; i < ROWS; i++) {
        const int r = r0 + i * PASS + (int)threadIdx.x / LPR;
        if (r < job.rows) store(r, ref[i], sum[i], o[i]);
      }
    }
    return;
  }
  const int sub = lane / LPR;
  for (int r = chunk * kJoinWaves + wave; r < job.rows; r += chunks * kJoinWaves) {
    float ref = -INFINITY, sum = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
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
    for (; x0 + 8 * SIDE < n; x0 += 16 * SIDE) join(std::integral_constant<int, 16>{}, x0);
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
    if (sub == 0) store(r, ref, sum, o);
  }
}

// Workgroups of the launch: four rows each of the tiles that may be split, up
// to four for each CU, which run at once, and never fewer than those tiles.
inline int join_workgroups(const AttnArgs &a, int B) {
  const long long tiles = std::min<long long>(B, (1 + (long long)a.T * a.G / a.part_rows) * a.R * a.c.n_heads);
  return (int)std::min<long long>(std::max(B, 4 * num_cus()), tiles * ((a.part_rows + kJoinWaves - 1) / kJoinWaves));
}

}  // namespace k3
