// What the operators' C entry points share: statuses with a text, launch errors,
// alignment.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdarg>
#include <cstdio>

#include "wq_block_internal.hpp"

namespace wq::api {

constexpr int64_t kMaxDim = (int64_t)1 << 30;

inline wq_status fail(wq_status st, const char* fmt, ...) {
  char text[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  return wq::api_error(st, text);
}

inline wq_status launched(hipError_t e, const char* what) {
  if (e == hipErrorInvalidConfiguration) return fail(WQ_EUNSUPPORTED, "%s: more tiles than a launch holds", what);
  return e == hipSuccess ? wq::api_ok() : fail(WQ_EHIP, "%s launch: %s", what, hipGetErrorString(e));
}

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace wq::api
