// What the C ABI's source files share: the calling thread's error message,
// argument checks and workspace rounding (internal to libpoetx.so).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/poetx.h"

namespace poetx {

// message of the calling thread's most recent failure (poetx_last_error)
extern thread_local char g_err[512];
int32_t fail(int32_t st, const char* fmt, ...);
int32_t ok();
int32_t dev_fail(hipError_t e, const char* where);

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline size_t es_of(int act) { return act == POETX_BF16 ? 2 : 4; }
inline size_t align_up(size_t x) { return (x + 255) & ~size_t(255); }

#define NEED_PTR(p)                                                                  \
  do {                                                                               \
    if (!(p)) return fail(POETX_ERR_ARG, "%s: null pointer '%s'", fn, #p);           \
    if (!aligned16(p)) return fail(POETX_ERR_ARG, "%s: '%s' not 16-byte aligned", fn, #p); \
  } while (0)
#define OPT_PTR(p)                                                                   \
  do {                                                                               \
    if ((p) && !aligned16(p))                                                        \
      return fail(POETX_ERR_ARG, "%s: '%s' not 16-byte aligned", fn, #p);            \
  } while (0)

}  // namespace poetx
