// What the files of the C ABI share: the thread-local error text, the checks'
// helpers and the guard that keeps C++ exceptions inside.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/nvfp4.h"

namespace nvfp4 {

inline thread_local char g_last_error[512] = "";

inline int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
  va_end(ap);
  return status;
}

inline int ok() {
  g_last_error[0] = '\0';
  return NVFP4_OK;
}

inline int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(NVFP4_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }
inline bool aligned4(const void* p) { return aligned(p, 4); }

constexpr int64_t kMaxDim = int64_t(1) << 30;

}  // namespace nvfp4

#define NVFP4_TRY(expr)              \
  do {                               \
    int s_ = (expr);                 \
    if (s_ != NVFP4_OK) return s_;   \
  } while (0)

#define NVFP4_GUARD_BEGIN try {
#define NVFP4_GUARD_END                                                           \
  }                                                                               \
  catch (...) {                                                                   \
    return nvfp4::fail(NVFP4_ERR_ARG, "internal error: unexpected C++ exception"); \
  }
