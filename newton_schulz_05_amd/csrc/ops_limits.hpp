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

// ---- tensors that the caches do not hold ----
// Inputs beyond kStreamIn bytes are read past the caches: the last-level cache
// holds 256 MB, so that nobody finds them there again (logits of 8192 x 65536
// bf16, forward 162 us against 185; but 8192 x 5000, which the backward pass
// finds there, takes it 34 us instead of 29).  Outputs beyond kStreamOut bytes are
// written past them.  With a copy of the output right behind the call: gradient
// of 2048 x 32768 bf16 102 us against 118, 515 x 50021 fp32 70.6 and 70.8 (alone
// 27.8 and 36.8), but 1536 x 32768 77 and 75, 1024 x 32768 56 and 47.
constexpr int64_t kStreamIn = int64_t(256) << 20, kStreamOut = int64_t(96) << 20;

// ---- norm and rotation of query and key heads ----
constexpr int64_t kHeadMaxDim = 512;  // a head's row is held by at most one wave
constexpr int64_t kHeadMaxRows = 0x7fffffff;
constexpr int kHeadThreads = 256;

// Quotients of numbers r below 2^31 by d: floor(r mul / 2^(32 + shift)), with mul =
// ceil(2^(31 + s) / d) and shift = s - 1 for 2^(s - 1) < d <= 2^s.  mul d exceeds
// 2^(31 + s) by less than 2^s, so that r times the excess stays below 2^(31 + s)
// and the quotient below the next whole number.  d = 1 is left to the caller.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(int64_t d) {
  FastDiv f{uint32_t(d), 0, 0};
  if (d > 1) {
    int s = 1;
    while ((int64_t(1) << s) < d) ++s;
    f.mul = uint32_t(((uint64_t(1) << (31 + s)) + uint64_t(d) - 1) / uint64_t(d));
    f.shift = uint32_t(s - 1);
  }
  return f;
}

// Lanes that share one head's row, 16 elements each.  Pairs that lie rot / 2
// apart are one lane's: 8 elements of the first half of the turned ones with
// those of the second half, then the elements that are not turned, 16 a lane.
inline int head_lanes(int dim, int rot, bool interleaved) {
  const int need = interleaved || rot == 0 ? (dim + 15) / 16 : (rot / 2 + 7) / 8 + (dim - rot + 15) / 16;
  int lanes = 4;
  while (lanes < need) lanes *= 2;
  return lanes;
}

// The most lanes it gives: interleaved pairs fill 16 elements a lane, and so do whole
// pieces of 8; other segments, halves and the rest, may leave part of a lane empty.
constexpr int head_most_lanes(bool interleaved, bool whole, int size) {
  return interleaved || (whole && size == 2) ? int(kHeadMaxDim) / 16 : int(kHeadMaxDim) / 8;
}

// Workgroups of the backward pass, one partial sum of dgamma each: a fixed number
// in all, queries and keys in proportion to their rows.
constexpr int kHeadMaxParts = 1024;
struct HeadSplit {
  int q, k;
};
inline HeadSplit head_split(int64_t rows_q, int64_t rows_k) {
  // 32 rows a workgroup at least, whatever the lanes of a row (64 tokens of 32 + 8
  // heads of 128 bf16 7.1 us, 8.0 with 64 rows)
  const int64_t all = rows_q + rows_k, parts = std::min<int64_t>(kHeadMaxParts, (all + 31) / 32);
  HeadSplit s{0, 0};
  if (rows_k > 0) s.k = int(std::max<int64_t>(1, parts * rows_k / all));
  if (rows_q > 0) s.q = int(std::max<int64_t>(1, parts - s.k));  // each at most kHeadMaxParts
  return s;
}

// ---- token log-probabilities ----
constexpr int64_t kLogpMaxVocab = int64_t(1) << 24;
// Workgroups that share one row of the forward pass, whose parts a second launch
// joins: for few rows above 65536 words.  A row of 65536 bf16 takes one workgroup
// 6.9 us and several 5.2, but their second launch costs the host 3 us more; one of
// 131072 takes 10.4 and 5.2; 128 rows of 65536 8.4 and 9.2.
constexpr int kLogpMaxParts = 64;
constexpr int64_t kLogpFewRows = 512;
inline int logp_parts(int64_t rows, int64_t vocab) {
  if (rows >= kLogpFewRows || vocab <= 65536) return 1;
  const int64_t want = (kLogpFewRows + rows - 1) / std::max<int64_t>(rows, 1);
  return int(std::min<int64_t>({want, (vocab + 4095) / 4096, int64_t(kLogpMaxParts)}));
}

// ---- losses ----
constexpr int64_t kLossMaxTokens = int64_t(1) << 40;
constexpr int64_t kPrefMaxPairs = int64_t(1) << 20;
constexpr int kPolicyMaxParts = 256, kPrefMaxChunks = 64;
// One workgroup up to four tokens a thread (4096: 7.2 us, 6.1 with two launches,
// which cost the host 4 us more).
inline int policy_parts(int64_t tokens) {
  return tokens <= 4096 ? 1 : int(std::min<int64_t>((tokens + 1023) / 1024, kPolicyMaxParts));
}
// The preference loss by one workgroup, a wave a sequence; else each sequence by
// 2^shift workgroups in two launches, which cost the host 4 us more.  A pair of
// 2 x 100 tokens 3.8 us and 5.4, 2 x 2000 7.2 and 5.5, 2 x 4096 12.3 and 5.8.
constexpr int64_t kPrefLonePairs = 8, kPrefLoneTokens = 4096;
inline bool pref_lone(int64_t tokens, int64_t pairs) { return pairs <= kPrefLonePairs && tokens <= kPrefLoneTokens; }
inline int pref_shift(int64_t tokens, int64_t pairs) {
  const int64_t each = tokens / std::max<int64_t>(2 * pairs, 1);
  int s = 0;
  while ((1 << s) < kPrefMaxChunks && (int64_t(512) << s) < each) ++s;
  return s;
}

}  // namespace muon
