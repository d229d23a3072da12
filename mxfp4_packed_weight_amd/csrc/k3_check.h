// Argument checks that the step's entry points share (k3_kv_abi.hip,
// k3_step_abi.hip): each refuses with a message that names the call.
#pragma once

#include <stdarg.h>
#include <stdio.h>

#include "k3_internal.h"

namespace k3 {

constexpr int kMaxTokens = 1 << 20;

inline k3_status refuse(k3_status s, const char *fmt, ...) {
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

k3_status check_cache(const char *fn, const k3_kv_cache *c);
k3_status check_rows(const char *fn, const char *what, int64_t stride, int T, int heads, int D);
k3_status check_tokens(const char *fn, int T, int Hq, int n_heads);
k3_status check_table(const char *fn, int R, int blocks, int page_size);

}  // namespace k3
