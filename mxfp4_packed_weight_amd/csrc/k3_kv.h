// Internal declarations of the paged key/value cache calls (k3_kv_*.hip).
#pragma once

#include "k3_internal.h"

namespace k3 {

struct KvPlanArgs {
  const int32_t *ctx, *new_, *parents, *held, *ring_state;
  int32_t *ring, *table, *held_out, *ring_out, *cu, *kv_lens, *slots, *positions, *mask, *status;
  int R, T, n_pages, page, blocks, words;
};
hipError_t launch_kv_plan(const KvPlanArgs &a, hipStream_t s);

struct QkArgs {
  const uint16_t *q, *k, *v, *wq, *wk;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const float *inv_freq;
  const int32_t *positions, *slots;
  uint16_t *q_out;
  k3_kv_cache c;
  float eps;
  int dtype, T, Hq, rot, interleaved;
};
hipError_t launch_qk_norm_rope(const QkArgs &a, hipStream_t s);

struct KvCommitArgs {
  k3_kv_cache c;
  int64_t layer_stride;
  const int32_t *table, *ctx, *kv_lens, *accepted, *n_accepted;  // kv_lens may be null
  int32_t *ctx_out;
  int layers, blocks, most, R;
};
hipError_t launch_kv_commit(const KvCommitArgs &a, hipStream_t s);

struct KvAppendArgs {
  const uint16_t *k, *v;
  int64_t k_stride, v_stride;
  k3_kv_cache c;
  uint8_t *k_exp, *v_exp;
  const int32_t *table, *cu, *kv_lens;
  int dtype, T, blocks, R;
};
hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t s);

// Attention: q and out are 16-bit rows of the type the kernel is built for.
struct AttnArgs {
  const uint16_t *q;
  int64_t q_stride, out_stride;
  k3_kv_cache c;
  const int32_t *table, *cu, *kv_lens, *mask;
  uint16_t *out;
  float *lse, *part;  // part: the partial results of split tiles, of up to part_rows rows
  float scale;
  int dtype, T, Hq, G, blocks, R, words, part_rows;
  // x / d for x < 2^31 is umulhi(2x, magic) >> shift: places by page_size, rows by G
  uint32_t page_magic, group_magic;
  int page_shift, group_shift;
  int window, sinks;  // a row at position x sees places below sinks, and above x - window (window >= 1)
  const uint8_t *k_exp, *v_exp;  // of pages and heads, or null
  int whole;        // no tile is split, and nothing joined
  int slope;        // 16 tile_rows / G
  double inv_groups;  // 1 / workgroups of the launch
};
int attn_tile_rows(int T, int G, int R, int D);
int attn_workgroups(int tile_rows, int D);
size_t attn_workspace_bytes(int T, int Hq, int n_heads, int D);
// The variants of the attention kernels: every place that causality or a mask
// allows; those in a window; the same over a cache with exponents.
constexpr int kAllPlaces = 0, kWindow = 1, kBlocks = 2;
hipError_t launch_attention(const AttnArgs &a, int mode, hipStream_t s);

}  // namespace k3
