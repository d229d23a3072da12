// Commit of the accepted paths: rows of keys and values move down within a
// request's pages, in every layer.
//
// A table keeps the ids of pages that a request has given back, and they may
// be another's by then; kv_lens says how far a step's places are its own.
//
// One workgroup per request and layer; each thread owns one 16-byte column of
// a row (heads x keys and values) and takes it through the path's rows, eight
// rows in flight. accepted ascends strictly, so accepted[i] >= i: a row that
// is written was read before, or is read by no later step, and since a
// thread's columns are its own nothing has to be kept apart. Each moved row
// is read once and written once; rows that stay are not written (their load
// reads the first row of page 0). 64 paths of up to 6 nodes through 48 layers,
// 74 MB: 21 us (15 at a copy's rate; runs of layers to a workgroup are no
// faster).
#include "k3_kv.h"

namespace k3 {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kCommitThreads = 256;
constexpr int kInFlight = 8;

// Byte offset of a place's first row, -1 if it has no page.
__device__ __forceinline__ int64_t place_offset(const KvCommitArgs &a, const int32_t *table_row, int64_t p, int es) {
  const int64_t b = p / a.c.page_size;
  const int page = b < a.blocks ? table_row[b] : -1;
  if (page < 0 || page >= a.c.n_pages) return -1;
  return (page * a.c.page_stride + (p - b * a.c.page_size) * a.c.slot_stride) * es;
}

__global__ __launch_bounds__(kCommitThreads) void kv_commit_kernel(KvCommitArgs a, int row16) {
  __shared__ int64_t src[K3_MAX_ACCEPTED], dst[K3_MAX_ACCEPTED];  // byte offsets
  __shared__ int bad;
  const int r = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
  const int n = a.n_accepted[r], ctx = a.ctx[r];
  const int len = a.kv_lens ? a.kv_lens[r] : INT32_MAX;
  const int es = a.c.dtype == K3_E4M3 ? 1 : 2;
  const int32_t *row = a.table + (size_t)r * a.blocks, *acc = a.accepted + (size_t)r * a.most;
  if (tid == 0) bad = n < 0 || n > a.most || ctx < 0;
  __syncthreads();
  const int todo = bad ? 0 : n;
  __syncthreads();
  for (int i = tid; i < todo; i += kCommitThreads) {
    const int from = acc[i], before = i ? acc[i - 1] : -1;
    int64_t s_at = -1, d_at = -1;
    // before >= -1: ascending, and not below zero; then i <= from, so that one
    // look at the request's places is enough
    if (from > before && (int64_t)ctx + from < len) {
      s_at = place_offset(a, row, (int64_t)ctx + from, es);
      d_at = from == i ? s_at : place_offset(a, row, (int64_t)ctx + i, es);
    }
    if (s_at < 0 || d_at < 0) bad = 1;
    src[i] = from == i ? 0 : s_at;
    dst[i] = from == i ? 0 : d_at;
  }
  __syncthreads();
  // (all n places are in the table's row, so the sum is at most 2^30)
  if (layer == 0 && tid == 0) a.ctx_out[r] = bad ? ctx : ctx + n;
  if (bad) return;
  const int per_head = row16, cols = a.c.n_heads * per_head;
  const int64_t base = layer * a.layer_stride * es;
  for (int c = tid; c < 2 * cols; c += kCommitThreads) {
    char *p = (char *)(c < cols ? a.c.k : a.c.v) + base;
    const int x = c < cols ? c : c - cols, h = x / per_head;
    p += h * a.c.head_stride * es + (x - h * per_head) * 16;
    for (int i0 = 0; i0 < todo; i0 += kInFlight) {
      u32x4 v[kInFlight];
#pragma unroll
      for (int i = 0; i < kInFlight; i++)
        v[i] = *(const u32x4 *)(p + (i0 + i < todo ? src[i0 + i] : 0));
#pragma unroll
      for (int i = 0; i < kInFlight; i++)
        if (i0 + i < todo && src[i0 + i] != dst[i0 + i]) *(u32x4 *)(p + dst[i0 + i]) = v[i];
    }
  }
}

}  // namespace

hipError_t launch_kv_commit(const KvCommitArgs &a, hipStream_t s) {
  const int row16 = a.c.head_dim * (a.c.dtype == K3_E4M3 ? 1 : 2) / 16;
  kv_commit_kernel<<<dim3(a.R, a.layers), kCommitThreads, 0, s>>>(a, row16);
  return hipGetLastError();
}

}  // namespace k3
