// Argument checks shared by the C entry points of the layers, the products by group and the
// optimiser.
#pragma once
#include <hip/hip_runtime.h>

#include <limits>
#include <string>

#include "internal.hpp"

namespace tpc {

inline tp_status fail(const char* where, const char* what, tp_status code = TP_ERR_ARG) {
  return set_error(code, std::string(where) + ": " + what);
}

// No exception leaves a C entry point.
template <typename F>
tp_status guarded(F&& f) noexcept {
  try {
    return f();
  } catch (...) {
    return TP_ERR_HIP;
  }
}

inline bool known(int32_t dtype) { return dtype == TP_F32 || dtype == TP_BF16; }
inline int64_t size_of(int32_t dtype) { return dtype == TP_F32 ? 4 : 2; }
inline bool aligned(const void* p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(to - 1)) == 0; }

inline bool bad_stride(int64_t stride, int64_t cols, int64_t rows) {
  return stride < cols || (rows > 0 && stride > std::numeric_limits<int64_t>::max() / 8 / rows);
}

// the status of a launch that may be refused for its size
inline tp_status launched(const char* where, hipError_t e, const char* too_large = "too many rows for one launch") {
  if (e == hipErrorInvalidConfiguration) return fail(where, too_large, TP_ERR_OVERFLOW);
  return e == hipSuccess ? TP_OK : hip_error(e, (std::string(where) + " launch").c_str());
}

}  // namespace tpc
