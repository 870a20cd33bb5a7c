// What the C entry points of the operators around the layer check the same way.
#pragma once

#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../../include/wtconv_block.h"
#include "../wtconv_launch.h"

namespace wtb {
namespace api {

inline wtconv_status_t fail(wtconv_status_t st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline wtconv_status_t fail(wtconv_status_t st, const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  wt::set_last_error(msg);
  return st;
}

inline int esize(int dtype) { return dtype == WTCONV_F32 ? 4 : 2; }

inline wtconv_status_t pointer(const void* p, const char* name, int align, bool nullable = false) {
  if (!p) return nullable ? WTCONV_OK : fail(WTCONV_ERR_INVALID_ARG, "%s is NULL", name);
  if ((uintptr_t)p % align) return fail(WTCONV_ERR_MISALIGNED, "%s is not %d-byte aligned", name, align);
  return WTCONV_OK;
}

inline wtconv_status_t workspace(const void* ws, size_t given, size_t need) {
  if (need == 0) return WTCONV_OK;
  if (!ws || given < need) return fail(WTCONV_ERR_WORKSPACE, "workspace of %zu B given, %zu B needed", ws ? given : 0, need);
  if ((uintptr_t)ws % 256) return fail(WTCONV_ERR_MISALIGNED, "workspace is not 256-byte aligned");
  return WTCONV_OK;
}

#define TRY(e)                                       \
  do {                                               \
    const wtconv_status_t st_ = (e);                 \
    if (st_ != WTCONV_OK) return st_;                \
  } while (0)

// Elements of the widest access (at most 16 bytes) that an address and its
// strides allow.
inline int widest(int es, const void* p, long long sample, long long row, long long n, long long s) {
  int v = 16 / es;
  while (v > 1 && ((uintptr_t)p % (v * es) || (s > 1 && row % v) || (n > 1 && sample % v))) v >>= 1;
  return v;
}

inline wtconv_status_t cuda_status(cudaError_t e, const char* name) {
  return e == cudaSuccess ? WTCONV_OK : fail(WTCONV_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
}

}  // namespace api
}  // namespace wtb
