// Internal declarations of the step's calls beside the cache (k3_norm.hip,
// k3_kv_append.hip, k3_logprobs.hip).
#pragma once

#include "k3_internal.h"

namespace k3 {

struct NormArgs {
  const uint16_t *x, *residual, *w;  // residual may be null
  uint16_t *sum, *y;                 // may be null
  uint8_t *y8;                       // may be null
  float *scales;
  int64_t x_stride, residual_stride, sum_stride, y_stride, y8_stride;
  float eps;
  int dtype, T, hidden, group;
};
hipError_t launch_add_rms_norm(const NormArgs &a, hipStream_t s);

// A part of a row, or its joined parts: the reference value m, sum of
// exp((x - m) beta), sum of exp((x - m) beta) (x - m), and lists of the largest.
struct LogprobArgs {
  const void *logits;
  int64_t stride;
  const int32_t *tokens;
  float *logprob, *entropy, *lse;  // may be null (tokens with logprob)
  int32_t *top;
  float *top_logprob;
  float *part;  // [T][parts] of part_words(k) words
  float beta;
  int dtype, T, V, k, parts;
};
int logprob_parts(int T, int V);
size_t logprob_workspace_parts(int T, int V);  // for up to T rows
inline size_t logprob_part_words(int k) { return 4 + 2 * (size_t)k; }
hipError_t launch_token_logprobs(const LogprobArgs &a, hipStream_t s);

}  // namespace k3
