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
  int slope;        // 16 tile_rows / G
  double inv_groups;  // 1 / workgroups of the launch
};
int attn_tile_rows(int T, int G, int R, int D);
int attn_workgroups(int tile_rows, int D);
size_t attn_workspace_bytes(int T, int Hq, int n_heads, int D);
hipError_t launch_tree_attention(const AttnArgs &a, hipStream_t s);

}  // namespace k3
