// What the training operators' entry points share: descriptions of their
// tensors, and how errors leave them.
#pragma once

#include <hip/hip_runtime.h>

#include <string>
#include <vector>

#include "../../include/muon.h"
#include "launch.hpp"
#include "ops.hpp"
#include "validate_ops.hpp"

#define MUON_TRY(call)                                   \
  do {                                                   \
    if (const muon_status s_ = (call); s_ != MUON_OK) return s_; \
  } while (0)

namespace muon {
namespace api {

inline int64_t elem(muon_dtype dt) { return dt == MUON_BF16 ? 2 : 4; }

inline Operand matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, muon_dtype dt,
                      bool written, bool optional = false) {
  return {name, p, rows, cols * elem(dt), ld * elem(dt), int(elem(dt)), written, optional};
}
// n elements of `size` bytes.
inline Operand vec(const char* name, const void* p, int64_t n, int64_t size, bool written, bool optional = false) {
  return {name, p, n > 0 ? 1 : 0, n * size, n * size, int(size), written, optional};
}

inline muon_status launched(hipError_t e) {
  if (e == hipSuccess) return MUON_OK;
  return api_fail(MUON_ERR_HIP, std::string("kernel launch failed: ") + hipGetErrorString(e));
}

// No C++ exception (an out-of-memory std::bad_alloc of the argument lists)
// leaves a C entry point.
template <typename F> muon_status guarded(F f) {
  try {
    std::string d;
    const muon_status s = f(&d);
    return s == MUON_OK || d.empty() ? s : api_fail(s, d);
  } catch (...) {
    return MUON_ERR_INVALID_ARG;
  }
}

}  // namespace api
}  // namespace muon
