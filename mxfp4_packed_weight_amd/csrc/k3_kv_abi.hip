// C ABI of the paged key/value cache: argument checks and launches. As in
// k3_abi.hip every check happens before the first launch.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>

#include "k3_attn.h"

namespace k3 {

hipError_t launch_attn_bf16(const AttnArgs &a, hipStream_t s);
hipError_t launch_attn_bf16_e4m3(const AttnArgs &a, hipStream_t s);
hipError_t launch_attn_f16(const AttnArgs &a, hipStream_t s);
hipError_t launch_attn_f16_e4m3(const AttnArgs &a, hipStream_t s);

// Rows per tile: up to 32 rows of an average request (16 at a head of 256) go
// to the streaming kernel, more to the tiled kernel. Streaming (its better
// tile) against tiled, 32 requests of 8192 places, 8 query heads to a key head,
// us:
//   rows                           16          32          48
//   8 key heads of 128, bf16    174 / 193   177 / 193   340 / 194
//   8 of 128, e4m3               99 / 138   119 / 138   223 / 150
//   8 of 64, bf16                95 / 105   104 / 105   198 / 106
//   4 of 256, bf16              178 / 203   307 / 205   501 / 209
//   8 of 256, bf16              335 / 366   659 / 366   984 / 368
// The lengths are on the device, so the average is all that the rule sees, and
// R counts requests without tokens too. A batch of unlike requests can
// therefore be slower than with the other kernel, since each streaming tile of
// a long request reads all of its keys again. 8 key heads of 128, ragged
// contexts of up to 8191, streaming as the rule's tile has it / tiled:
//   255 tokens, one chunk of 512, 8 heads to a key head, bf16   1373 / 785
//   the same, e4m3                                              1160 / 818
//   255 tokens, one chunk of 255, bf16                           934 / 775
//   255 tokens, one chunk of 255, e4m3                           614 / 759
//   255 tokens, one tree of 64, bf16                             802 / 783
//   63 tokens, one chunk of 512, bf16 (the rule: tiled)          654 / 277
// and 16 key heads, a head each, one chunk of 2048 among 256 requests of which
// the others have no tokens: 168 / 51 over no context, 1230 / 164 over 8192.
// A caller that knows its batch puts the long requests last and makes two
// calls, of the first requests' tokens alone and of the last requests.
int attn_tile_rows(int T, int G, int R, int D) {
  const long long rows = ((long long)T * G + R - 1) / R;
  if (rows <= 16) return 16;
  if (D == 256) return 128;
  return rows <= 32 ? 32 : 256;
}

// Two workgroups of the streaming kernel's 16-row tiles fit on a CU (one at a
// head of 256), one of the others.
int attn_workgroups(int tile_rows, int D) {
  const int cus = std::min(num_cus(), kMaxWorkgroups / 2);
  return tile_rows == 16 && D < 256 ? 2 * cus : cus;
}

static int attn_part_rows(int tile_rows, int T, int G) { return (int)std::min((long long)tile_rows, (long long)T * G); }

size_t attn_workspace_bytes(int T, int Hq, int n_heads, int D) {
  // R is not known here: any tile up to the one request's may be taken
  const int G = Hq / n_heads, largest = attn_tile_rows(T, G, 1, D);
  size_t rows = 0;
  for (int r : {16, 32, 128, 256})
    if (r <= largest) rows = std::max(rows, (size_t)2 * attn_workgroups(r, D) * attn_part_rows(r, T, G));
  return rows * (D + 2) * sizeof(float) + kMaxWorkgroups * sizeof(JoinJob);
}

hipError_t launch_tree_attention(const AttnArgs &a, hipStream_t s) {
  const bool f8 = a.c.dtype == K3_E4M3;
  if (a.dtype == K3_BF16) return f8 ? launch_attn_bf16_e4m3(a, s) : launch_attn_bf16(a, s);
  return f8 ? launch_attn_f16_e4m3(a, s) : launch_attn_f16(a, s);
}

namespace {

constexpr int kMaxTokens = 1 << 20;

k3_status refuse(k3_status s, const char *fmt, ...) {
  char text[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof text, fmt, ap);
  va_end(ap);
  set_error("%s", text);
  return s;
}

#define KV_PTR(p, align)                                                                       \
  do {                                                                                         \
    if (!(p)) return refuse(K3_ERR_ARG, "%s: %s is NULL", fn, #p);                             \
    if ((uintptr_t)(p) % (align))                                                              \
      return refuse(K3_ERR_ARG, "%s: %s is not %d-byte aligned", fn, #p, (int)(align));        \
  } while (0)
// A pointer that may be NULL.
#define KV_OPT(p, align)                                                                       \
  do {                                                                                         \
    if ((uintptr_t)(p) % (align))                                                              \
      return refuse(K3_ERR_ARG, "%s: %s is not %d-byte aligned", fn, #p, (int)(align));        \
  } while (0)
#define KV_NEED(cond, ...)                                     \
  do {                                                         \
    if (!(cond)) return refuse(K3_ERR_CONFIG, __VA_ARGS__);    \
  } while (0)

k3_status check_cache(const char *fn, const k3_kv_cache *c) {
  if (!c) return refuse(K3_ERR_ARG, "%s: cache is NULL", fn);
  KV_PTR(c->k, 16);
  KV_PTR(c->v, 16);
  KV_OPT(c->k_scale, 4);
  KV_OPT(c->v_scale, 4);
  KV_NEED(c->dtype == K3_BF16 || c->dtype == K3_F16 || c->dtype == K3_E4M3,
          "%s: cache dtype=%d is none of K3_BF16, K3_F16, K3_E4M3", fn, c->dtype);
  KV_NEED(c->dtype == K3_E4M3 || (!c->k_scale && !c->v_scale), "%s: only an e4m3 cache has scales", fn);
  KV_NEED(c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256,
          "%s: head_dim=%d is none of 64, 128, 256", fn, c->head_dim);
  KV_NEED(c->n_heads >= 1 && c->n_heads <= K3_MAX_HEADS, "%s: n_heads=%d outside [1, %d]", fn, c->n_heads,
          K3_MAX_HEADS);
  KV_NEED(c->n_pages >= 1 && c->page_size >= 1 && (int64_t)c->n_pages * c->page_size <= INT32_MAX,
          "%s: n_pages=%d, page_size=%d: both at least 1, their product below 2^31", fn, c->n_pages, c->page_size);
  // (one page, slot or head has no use for its stride)
  const int64_t unit = c->dtype == K3_E4M3 ? 16 : 8;
  const int64_t strides[3] = {c->page_stride, c->slot_stride, c->head_stride};
  const int32_t sizes[3] = {c->n_pages, c->page_size, c->n_heads};
  for (int i = 0; i < 3; i++)
    KV_NEED(sizes[i] == 1 || (strides[i] >= c->head_dim && strides[i] % unit == 0),
            "%s: cache strides %lld, %lld, %lld must be multiples of 16 bytes and at least a row of %d", fn,
            (long long)strides[0], (long long)strides[1], (long long)strides[2], c->head_dim);
  return K3_OK;
}

k3_status check_rows(const char *fn, const char *what, int64_t stride, int T, int heads, int D) {
  KV_NEED(T <= 1 || (stride % 8 == 0 && stride >= (int64_t)heads * D),
          "%s: %s=%lld must be a multiple of 8, and at least the %lld of its dense heads", fn, what,
          (long long)stride, (long long)heads * D);
  return K3_OK;
}

k3_status check_tokens(const char *fn, int T, int Hq, int n_heads) {
  KV_NEED(T >= 0 && T <= kMaxTokens, "%s: T=%d outside [0, %d]", fn, T, kMaxTokens);
  KV_NEED(Hq >= 1 && Hq <= K3_MAX_HEADS && Hq % n_heads == 0,
          "%s: Hq=%d must be a multiple of n_heads=%d (<= %d)", fn, Hq, n_heads, K3_MAX_HEADS);
  return K3_OK;
}

k3_status check_table(const char *fn, int R, int blocks, int page_size) {
  KV_NEED(R >= 1 && R <= K3_MAX_REQUESTS, "%s: R=%d outside [1, %d]", fn, R, K3_MAX_REQUESTS);
  KV_NEED(blocks >= 1 && (int64_t)blocks * page_size <= 1 << 30,
          "%s: blocks=%d, page_size=%d: at least one block, at most 2^30 places", fn, blocks, page_size);
  return K3_OK;
}

}  // namespace

}  // namespace k3

using namespace k3;

extern "C" {

k3_status k3_kv_plan(const int32_t *ctx, const int32_t *new_, const int32_t *parents, int R, int T, int n_pages,
                     int page_size, int blocks, const int32_t *held, int32_t *ring, const int32_t *ring_state,
                     int32_t *table, int32_t *held_out, int32_t *ring_out, int32_t *cu, int32_t *kv_lens,
                     int32_t *slots, int32_t *positions, int32_t *mask, int words, int32_t *status,
                     k3_stream_t stream) {
  const char *fn = "k3_kv_plan";
  KV_PTR(ctx, 4);
  KV_PTR(new_, 4);
  KV_OPT(parents, 4);
  KV_PTR(held, 4);
  KV_PTR(ring, 4);
  KV_PTR(ring_state, 4);
  KV_PTR(table, 4);
  KV_PTR(held_out, 4);
  KV_PTR(ring_out, 4);
  KV_PTR(cu, 4);
  KV_PTR(kv_lens, 4);
  KV_PTR(status, 4);
  KV_NEED(T >= 0 && T <= kMaxTokens, "%s: T=%d outside [0, %d]", fn, T, kMaxTokens);
  KV_NEED(n_pages >= 1 && page_size >= 1 && n_pages <= 1 << 30 && (int64_t)n_pages * page_size <= INT32_MAX,
          "%s: n_pages=%d, page_size=%d: both at least 1, their product below 2^31", fn, n_pages, page_size);
  if (k3_status s = check_table(fn, R, blocks, page_size)) return s;
  if (T) {
    KV_PTR(slots, 4);
    KV_PTR(positions, 4);
    if (parents) KV_PTR(mask, 4);
  }
  KV_NEED(!parents || (words >= 1 && words <= K3_MAX_TREE_WORDS), "%s: words=%d outside [1, %d]", fn, words,
          K3_MAX_TREE_WORDS);
  const int32_t *in[] = {ctx, new_, held, ring_state, parents};
  const int32_t *out[] = {ring, table, held_out, ring_out, cu, kv_lens, slots, positions, mask, status};
  for (const int32_t *o : out)
    for (const int32_t *i : in)
      KV_NEED(!o || o != i, "%s: an output is the same array as an input (only ring and table are updated in place)", fn);
  KvPlanArgs a = {};
  a.ctx = ctx;
  a.new_ = new_;
  a.parents = T ? parents : nullptr;
  a.held = held;
  a.ring_state = ring_state;
  a.ring = ring;
  a.table = table;
  a.held_out = held_out;
  a.ring_out = ring_out;
  a.cu = cu;
  a.kv_lens = kv_lens;
  a.slots = slots;
  a.positions = positions;
  a.mask = mask;
  a.status = status;
  a.R = R;
  a.T = T;
  a.n_pages = n_pages;
  a.page = page_size;
  a.blocks = blocks;
  a.words = words;
  return device_status(launch_kv_plan(a, stream), fn);
}

k3_status k3_qk_norm_rope(const void *q_in, int64_t q_stride, const void *k_in, int64_t k_stride, const void *v_in,
                          int64_t v_stride, int dtype, int T, int Hq, const void *wq, const void *wk, float eps,
                          const float *inv_freq, int rot, int interleaved, const int32_t *positions, void *q_out,
                          int64_t q_out_stride, const k3_kv_cache *cache, const int32_t *slots, k3_stream_t stream) {
  const char *fn = "k3_qk_norm_rope";
  if (k3_status s = check_cache(fn, cache)) return s;
  KV_NEED(dtype == K3_BF16 || dtype == K3_F16, "%s: dtype=%d is neither K3_BF16 nor K3_F16", fn, dtype);
  KV_NEED(cache->dtype == K3_E4M3 || cache->dtype == dtype, "%s: a cache of dtype=%d for rows of dtype=%d", fn,
          cache->dtype, dtype);
  if (k3_status s = check_tokens(fn, T, Hq, cache->n_heads)) return s;
  const int D = cache->head_dim;
  KV_NEED(rot >= 0 && rot <= D && rot % 16 == 0, "%s: rot=%d must be a multiple of 16 (<= head_dim=%d)", fn, rot, D);
  KV_NEED(eps >= 0.f && eps <= 3.0e38f, "%s: eps=%g must be finite and not negative", fn, eps);
  KV_PTR(wq, 16);
  KV_PTR(wk, 16);
  if (rot) KV_PTR(inv_freq, 4);
  if (T == 0) return K3_OK;
  KV_PTR(q_in, 16);
  KV_PTR(k_in, 16);
  KV_PTR(v_in, 16);
  KV_PTR(positions, 4);
  KV_PTR(q_out, 16);
  KV_PTR(slots, 4);
  if (k3_status s = check_rows(fn, "q_stride", q_stride, T, Hq, D)) return s;
  if (k3_status s = check_rows(fn, "k_stride", k_stride, T, cache->n_heads, D)) return s;
  if (k3_status s = check_rows(fn, "v_stride", v_stride, T, cache->n_heads, D)) return s;
  if (k3_status s = check_rows(fn, "q_out_stride", q_out_stride, T, Hq, D)) return s;
  KV_NEED(q_out != k_in && q_out != v_in, "%s: q_out is k_in or v_in", fn);
  KV_NEED(q_out != q_in || T == 1 || q_out_stride == q_stride, "%s: q_out is q_in, with q_out_stride=%lld for q_stride=%lld",
          fn, (long long)q_out_stride, (long long)q_stride);
  QkArgs a = {};
  a.q = (const uint16_t *)q_in;
  a.k = (const uint16_t *)k_in;
  a.v = (const uint16_t *)v_in;
  a.wq = (const uint16_t *)wq;
  a.wk = (const uint16_t *)wk;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.slots = slots;
  a.q_out = (uint16_t *)q_out;
  a.c = *cache;
  a.eps = eps;
  a.dtype = dtype;
  a.T = T;
  a.Hq = Hq;
  a.rot = rot;
  a.interleaved = interleaved;
  return device_status(launch_qk_norm_rope(a, stream), fn);
}

size_t k3_tree_attention_workspace_bytes(int T, int Hq, int n_heads, int head_dim) {
  const char *fn = "k3_tree_attention_workspace_bytes";
  if (n_heads < 1 || n_heads > K3_MAX_HEADS || (head_dim != 64 && head_dim != 128 && head_dim != 256)) {
    refuse(K3_ERR_CONFIG, "%s: n_heads=%d, head_dim=%d", fn, n_heads, head_dim);
    return 0;
  }
  if (check_tokens(fn, T, Hq, n_heads) != K3_OK) return 0;
  return attn_workspace_bytes(std::max(T, 1), Hq, n_heads, head_dim);
}

k3_status k3_tree_attention(const void *q, int64_t q_stride, int dtype, int T, int Hq, const k3_kv_cache *cache,
                            const int32_t *table, int blocks, const int32_t *cu, const int32_t *kv_lens, int R,
                            const int32_t *mask, int words, float scale, void *out, int64_t out_stride, void *ws,
                            size_t ws_bytes, float *lse, k3_stream_t stream) {
  const char *fn = "k3_tree_attention";
  if (k3_status s = check_cache(fn, cache)) return s;
  KV_NEED(dtype == K3_BF16 || dtype == K3_F16, "%s: dtype=%d is neither K3_BF16 nor K3_F16", fn, dtype);
  KV_NEED(cache->dtype == K3_E4M3 || cache->dtype == dtype, "%s: a cache of dtype=%d for rows of dtype=%d", fn,
          cache->dtype, dtype);
  if (k3_status s = check_tokens(fn, T, Hq, cache->n_heads)) return s;
  if (k3_status s = check_table(fn, R, blocks, cache->page_size)) return s;
  KV_NEED(!mask || (words >= 1 && words <= K3_MAX_TREE_WORDS), "%s: words=%d outside [1, %d]", fn, words,
          K3_MAX_TREE_WORDS);
  KV_NEED(isfinite(scale), "%s: scale=%g must be finite", fn, scale);
  KV_PTR(table, 4);
  KV_PTR(cu, 4);
  KV_PTR(kv_lens, 4);
  KV_OPT(mask, 4);
  KV_OPT(lse, 4);
  KV_PTR(ws, 16);
  if (T == 0) return K3_OK;
  KV_PTR(q, 16);
  KV_PTR(out, 16);
  const int D = cache->head_dim;
  if (k3_status s = check_rows(fn, "q_stride", q_stride, T, Hq, D)) return s;
  if (k3_status s = check_rows(fn, "out_stride", out_stride, T, Hq, D)) return s;
  KV_NEED(q != out, "%s: out is q", fn);
  const size_t need = attn_workspace_bytes(T, Hq, cache->n_heads, D);
  if (ws_bytes < need)
    return refuse(K3_ERR_MEMORY, "%s: workspace of %zu bytes is below the %zu bytes this call needs (give a larger "
                  "workspace; no size limit of the path is reached)", fn, ws_bytes, need);
  AttnArgs a = {};
  a.q = (const uint16_t *)q;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.c = *cache;
  a.table = table;
  a.cu = cu;
  a.kv_lens = kv_lens;
  a.mask = mask;
  a.out = (uint16_t *)out;
  a.lse = lse;
  a.part = (float *)ws;
  a.scale = scale;
  a.dtype = dtype;
  a.T = T;
  a.Hq = Hq;
  a.G = Hq / cache->n_heads;
  a.blocks = blocks;
  a.R = R;
  a.words = words;
  // x / d = (x * m) >> (31 + s) for x < 2^31: s = ceil(log2 d), m the next
  // integer above 2^(31 + s) / d (m < 2^32, and m d - 2^(31 + s) <= 2^s)
  auto divisor = [](int d, uint32_t *magic, int *shift) {
    int s = 0;
    while ((1ll << s) < d) s++;
    *shift = s;
    *magic = (uint32_t)(((uint64_t)1 << (31 + s)) / d + 1);
  };
  divisor(cache->page_size, &a.page_magic, &a.page_shift);
  divisor(a.G, &a.group_magic, &a.group_shift);
  const int tile_rows = attn_tile_rows(T, a.G, R, D);
  a.part_rows = attn_part_rows(tile_rows, T, a.G);
  a.slope = 16 * tile_rows / a.G;
  a.inv_groups = 1.0 / attn_workgroups(tile_rows, D);
  return device_status(launch_tree_attention(a, stream), fn);
}

static k3_status commit(const char *fn, const k3_kv_cache *cache, int layers, int64_t layer_stride,
                        const int32_t *table, int blocks, const int32_t *ctx, const int32_t *kv_lens,
                        const int32_t *accepted, const int32_t *n_accepted, int most, int R, int32_t *ctx_out,
                        k3_stream_t stream) {
  if (k3_status s = check_cache(fn, cache)) return s;
  if (k3_status s = check_table(fn, R, blocks, cache->page_size)) return s;
  KV_NEED(layers >= 1 && layers <= 65535, "%s: layers=%d outside [1, 65535]", fn, layers);
  KV_NEED(layers == 1 || (layer_stride > 0 && layer_stride % (cache->dtype == K3_E4M3 ? 16 : 8) == 0),
          "%s: layer_stride=%lld must be a positive multiple of 16 bytes", fn, (long long)layer_stride);
  KV_NEED(most >= 1 && most <= K3_MAX_ACCEPTED, "%s: most=%d outside [1, %d]", fn, most, K3_MAX_ACCEPTED);
  KV_PTR(table, 4);
  KV_PTR(ctx, 4);
  KV_PTR(accepted, 4);
  KV_PTR(n_accepted, 4);
  KV_PTR(ctx_out, 4);
  KV_NEED(ctx_out != ctx && ctx_out != kv_lens && ctx_out != n_accepted && ctx_out != accepted,
          "%s: ctx_out is the same array as an input", fn);
  KvCommitArgs a = {};
  a.c = *cache;
  a.layer_stride = layer_stride;
  a.table = table;
  a.ctx = ctx;
  a.kv_lens = kv_lens;
  a.accepted = accepted;
  a.n_accepted = n_accepted;
  a.ctx_out = ctx_out;
  a.layers = layers;
  a.blocks = blocks;
  a.most = most;
  a.R = R;
  return device_status(launch_kv_commit(a, stream), fn);
}

k3_status k3_kv_commit(const k3_kv_cache *cache, int layers, int64_t layer_stride, const int32_t *table, int blocks,
                       const int32_t *ctx, const int32_t *accepted, const int32_t *n_accepted, int most, int R,
                       int32_t *ctx_out, k3_stream_t stream) {
  return commit("k3_kv_commit", cache, layers, layer_stride, table, blocks, ctx, nullptr, accepted, n_accepted, most,
                R, ctx_out, stream);
}

k3_status k3_kv_commit_ex(const k3_kv_cache *cache, int layers, int64_t layer_stride, const int32_t *table, int blocks,
                          const int32_t *ctx, const int32_t *kv_lens, const int32_t *accepted,
                          const int32_t *n_accepted, int most, int R, int32_t *ctx_out, k3_stream_t stream) {
  const char *fn = "k3_kv_commit_ex";
  KV_PTR(kv_lens, 4);
  return commit(fn, cache, layers, layer_stride, table, blocks, ctx, kv_lens, accepted, n_accepted, most, R, ctx_out,
                stream);
}

}  // extern "C"
