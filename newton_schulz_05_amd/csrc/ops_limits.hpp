// Limits and work splits of the training operators that the argument checks,
// the workspace sizes and the launches share.  No HIP here: the host tests
// build it with g++.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace muon {

constexpr int64_t kNormMaxCols = 32768;  // a row is held by one workgroup
constexpr int64_t kRouteMaxExperts = 1024;
constexpr int32_t kRouteMaxK = 16;       // a 16-lane group keeps one choice per lane

// Threads that share one row of a norm.  A thread holds one or two vectors of
// 8 elements of it, four beyond 16384 columns.
constexpr int norm_row_threads(int64_t cols) {
  return cols <= 128 ? 16 : cols <= 1024 ? 64 : cols <= 4096 ? 256 : cols <= 8192 ? 512 : 1024;
}
// Threads of a backward workgroup.
constexpr int norm_bwd_threads(int64_t cols) { return cols <= 8192 ? 512 : 1024; }

// Workgroups of the backward pass, each of which leaves one partial sum of
// the gradients of gamma and beta: at most two for each of 256 compute units
// (a fixed number, so that results do not depend on the device's).
constexpr int kNormMaxParts = 512;
inline int64_t norm_bwd_parts(int64_t rows, int64_t cols) {
  const int64_t per = norm_bwd_threads(cols) / norm_row_threads(cols);
  return std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, kNormMaxParts));
}

// Lanes that share one token of the router: each holds `per` experts.
constexpr int route_lanes(int64_t experts) { return experts <= 8 ? 8 : 16; }
constexpr int kRouteThreads = 256;

// Workgroups of the router's forward pass (one partial sum each).
inline int64_t route_parts(int64_t rows, int64_t experts) {
  const int64_t per = kRouteThreads / route_lanes(experts);
  return std::min<int64_t>((rows + per - 1) / per, 256);
}

}  // namespace muon
