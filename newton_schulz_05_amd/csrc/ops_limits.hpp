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

constexpr int64_t kOpsMaxGrid = 1 << 20;  // workgroups of a launch; a kernel loops over what is left

// Split of a norm's backward pass: threads that share a row, threads of a
// workgroup, and the number of partial sums of the gradients of gamma and beta,
// which a second launch joins.
//   up to 256 rows: no partial sums; one launch, whose last workgroups sum 64
//     columns each over all rows (they read x and dy again, out of the cache:
//     64 x 1536 bf16 fused 2.9 us against 7.3 with two launches, 256 x 4096 5.7
//     against 10.2);
//   many rows: one partial sum a workgroup, 1024 threads on each of 256 compute
//     units (a fixed number, so that results do not depend on the device's),
//     or, for narrow rows, 256 threads as long as 256 such workgroups take all
//     rows at once;
//   beyond 20480 columns the sums have a kernel of their own, with 64 partial
//     sums of each strip of 2048 columns.
// A thread holds one vector of 8 elements of its row up to 8192 columns; then
// 512 threads three (up to 12288), 1024 two (16384), 512 five (20480), 1024
// three or four.  512 x 3 against 1024 x 2 gains where registers are short (fused
// fp32 7000 x 8200: 228 us against 264, 5000 x 12000 245 against 262) and is
// within 4 % elsewhere; 4000 x 16384 bf16 takes 89.0 us with 1024 x 2, 93.5 with
// 512 x 4; 3300 x 20000 bf16 98 us with 512 x 5, 133 with the sums apart (fused
// 194 and 203, but fused fp32, where 512 x 5 spills most, 423 and 389).
struct NormBwdSplit {
  int row_threads, threads, parts;
};
constexpr int kNormMaxParts = 256;
constexpr int64_t kNormFewRows = 256, kNormSumsHereCols = 20480;
inline NormBwdSplit norm_bwd_split(int64_t rows, int64_t cols) {
  NormBwdSplit s;
  s.row_threads = 8;
  while (s.row_threads < 1024 && s.row_threads * 8 < cols) s.row_threads *= 2;
  s.threads = s.row_threads <= 128 && rows <= int64_t(256 / s.row_threads) * kNormMaxParts ? 256 : 1024;
  const int64_t per = s.threads / s.row_threads, most = cols <= kNormSumsHereCols ? kNormMaxParts : 64;
  s.parts = rows <= kNormFewRows ? 0 : int(std::min<int64_t>((rows + per - 1) / per, most));
  return s;
}

// Lanes that share one token of the router: each holds `per` experts.
constexpr int route_lanes(int64_t experts) { return experts <= 8 ? 8 : 16; }
constexpr int kRouteThreads = 512, kRouteBwdThreads = 256;

// Workgroups of the router's forward pass (one partial sum each), a fixed number
// like the norm's: two for each of 256 compute units, one beyond 128 experts,
// where a partial sum costs more than the second workgroup hides (bf16, with
// 512 and 256: 65536 x 128 23.2 and 24.5 us, 16384 x 256 16.2 and 14.5).  One,
// and no second launch, for tokens that it takes in two steps.
constexpr int kRouteMaxParts = 512;
inline int64_t route_parts(int64_t rows, int64_t experts) {
  const int64_t per = kRouteThreads / route_lanes(experts), most = experts <= 128 ? kRouteMaxParts : kRouteMaxParts / 2;
  return rows <= 2 * per ? 1 : std::min<int64_t>((rows + per - 1) / per, most);
}

}  // namespace muon
