// C ABI of the step's calls beside the cache: argument checks and launches.
#include <math.h>

#include "k3_check.h"
#include "k3_step.h"

using namespace k3;

extern "C" {

k3_status k3_add_rms_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride, int dtype,
                          int T, int hidden, const void *w, float eps, void *sum, int64_t sum_stride, void *y,
                          int64_t y_stride, uint8_t *y8, int64_t y8_stride, float *scales, int group,
                          k3_stream_t stream) {
  const char *fn = "k3_add_rms_norm";
  KV_NEED(dtype == K3_BF16 || dtype == K3_F16, "%s: dtype=%d is neither K3_BF16 nor K3_F16", fn, dtype);
  KV_NEED(T >= 0 && T <= kMaxTokens, "%s: T=%d outside [0, %d]", fn, T, kMaxTokens);
  KV_NEED(hidden >= 8 && hidden <= K3_MAX_HIDDEN && hidden % 8 == 0,
          "%s: hidden=%d must be a multiple of 8 in [8, %d]", fn, hidden, K3_MAX_HIDDEN);
  KV_NEED(eps >= 0.f && eps <= 3.0e38f, "%s: eps=%g must be finite and not negative", fn, eps);
  if (y8) {
    const bool lanes = group == 32 || group == 64 || group == 128 || group == 256 || group == 512;
    KV_NEED(group == hidden || (lanes && hidden % group == 0),
            "%s: group=%d must be hidden=%d, or 32, 64, 128, 256 or 512 and divide it", fn, group, hidden);
  }
  KV_PTR(w, 16);
  if (T == 0) return K3_OK;
  KV_PTR(x, 16);
  KV_OPT(residual, 16);
  KV_OPT(sum, 16);
  KV_OPT(y, 16);
  KV_OPT(y8, 8);
  if (!y && !y8) return refuse(K3_ERR_ARG, "%s: both y and y8 are NULL", fn);
  if (y8) KV_PTR(scales, 4);
  if (k3_status s = check_rows(fn, "x_stride", x_stride, T, 1, hidden)) return s;
  if (residual)
    if (k3_status s = check_rows(fn, "residual_stride", residual_stride, T, 1, hidden)) return s;
  if (sum)
    if (k3_status s = check_rows(fn, "sum_stride", sum_stride, T, 1, hidden)) return s;
  if (y)
    if (k3_status s = check_rows(fn, "y_stride", y_stride, T, 1, hidden)) return s;
  if (y8)
    if (k3_status s = check_rows(fn, "y8_stride", y8_stride, T, 1, hidden)) return s;
  // in place: a row is read whole before any of it is written
  const void *in[] = {x, residual};
  const int64_t in_stride[] = {x_stride, residual_stride};
  for (int i = 0; i < 2; i++) {
    KV_NEED(!in[i] || !sum || sum != in[i] || T == 1 || sum_stride == in_stride[i],
            "%s: sum is an input, with sum_stride=%lld for %lld", fn, (long long)sum_stride, (long long)in_stride[i]);
    KV_NEED(!in[i] || !y || y != in[i] || T == 1 || y_stride == in_stride[i],
            "%s: y is an input, with y_stride=%lld for %lld", fn, (long long)y_stride, (long long)in_stride[i]);
    KV_NEED(!in[i] || !y8 || (const void *)y8 != in[i], "%s: y8 is an input", fn);
  }
  KV_NEED(!sum || (sum != y && sum != (void *)y8), "%s: sum is another output", fn);
  KV_NEED(!y || y != (void *)y8, "%s: y is y8", fn);
  NormArgs a = {};
  a.x = (const uint16_t *)x;
  a.residual = (const uint16_t *)residual;
  a.w = (const uint16_t *)w;
  a.sum = (uint16_t *)sum;
  a.y = (uint16_t *)y;
  a.y8 = y8;
  a.scales = scales;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.sum_stride = sum_stride;
  a.y_stride = y_stride;
  a.y8_stride = y8_stride;
  a.eps = eps;
  a.dtype = dtype;
  a.T = T;
  a.hidden = hidden;
  a.group = group;
  return device_status(launch_add_rms_norm(a, stream), fn);
}

static k3_status check_logprobs(const char *fn, int T, int V, int k) {
  KV_NEED(T >= 0 && T <= kMaxTokens, "%s: T=%d outside [0, %d]", fn, T, kMaxTokens);
  KV_NEED(V >= 1 && V <= 1 << 24, "%s: V=%d outside [1, 2^24]", fn, V);
  KV_NEED(k >= 0 && k <= K3_MAX_TOPK && k <= V, "%s: k=%d outside [0, min(%d, V=%d)]", fn, k, K3_MAX_TOPK, V);
  return K3_OK;
}

size_t k3_token_logprobs_workspace_bytes(int T, int V, int k) {
  if (check_logprobs("k3_token_logprobs_workspace_bytes", T, V, k) != K3_OK) return 0;
  return logprob_workspace_parts(T, V) * logprob_part_words(k) * sizeof(float);
}

k3_status k3_token_logprobs(const void *logits, int64_t stride, int dtype, int T, int V, float beta,
                            const int32_t *tokens, int k, float *logprob, float *entropy, float *lse, int32_t *top,
                            float *top_logprob, void *ws, size_t ws_bytes, k3_stream_t stream) {
  const char *fn = "k3_token_logprobs";
  KV_NEED(dtype == K3_BF16 || dtype == K3_F16 || dtype == K3_F32, "%s: dtype=%d is none of K3_BF16, K3_F16, K3_F32",
          fn, dtype);
  if (k3_status s = check_logprobs(fn, T, V, k)) return s;
  KV_NEED(beta >= 0x1p-20f && beta <= 0x1p20f, "%s: beta=%g outside [2^-20, 2^20]", fn, beta);
  if (T == 0) return K3_OK;
  KV_PTR(logits, dtype == K3_F32 ? 4 : 2);
  KV_NEED(T == 1 || stride >= V, "%s: stride=%lld is below V=%d", fn, (long long)stride, V);
  KV_OPT(tokens, 4);
  KV_OPT(logprob, 4);
  KV_OPT(entropy, 4);
  KV_OPT(lse, 4);
  if (!tokens != !logprob) return refuse(K3_ERR_ARG, "%s: tokens and logprob go together", fn);
  if (k) {
    KV_PTR(top, 4);
    KV_PTR(top_logprob, 4);
  }
  const size_t parts = logprob_parts(T, V), need = T * parts * logprob_part_words(k) * sizeof(float);
  if (parts > 1) {
    KV_PTR(ws, 16);
    if (ws_bytes < need)
      return refuse(K3_ERR_MEMORY, "%s: workspace of %zu bytes is below the %zu bytes this call needs (give a larger "
                    "workspace; no size limit of the path is reached)", fn, ws_bytes, need);
  }
  LogprobArgs a = {};
  a.logits = logits;
  a.stride = stride;
  a.tokens = tokens;
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.top = top;
  a.top_logprob = top_logprob;
  a.part = (float *)ws;
  a.beta = beta;
  a.dtype = dtype;
  a.T = T;
  a.V = V;
  a.k = k;
  a.parts = (int)parts;
  return device_status(launch_token_logprobs(a, stream), fn);
}

}  // extern "C"
