// Argument validation of the training operators' entry points (layer norm,
// dropout, router, query and key heads, token log-probabilities, losses).  Pure
// C++ (no HIP calls), like validate.hpp: each function returns MUON_OK, or an
// error status with `detail` filled, before anything is enqueued, and none of them
// touches device memory.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <string>
#include <utility>
#include <vector>

#include "../../include/muon.h"
#include "ops_limits.hpp"

namespace muon {

// One tensor argument: `rows` runs of `width` bytes, `pitch` bytes apart.
struct Operand {
  const char* name;
  const void* p;
  int64_t rows, width, pitch;
  int align;      // bytes
  bool written;
  bool optional;  // may be null
  // A tensor of heads also by its dimensions (batch, tokens, heads): entries, and
  // strides in bytes; each entry is `inner` bytes.  0 inner: no such tensor.
  int64_t n[3] = {0, 0, 0}, s[3] = {0, 0, 0}, inner = 0;
};

// Whether two operands share a byte.  Runs of one common pitch are compared
// by their place within the pitch, so that column slices of one buffer count
// as apart, and so are two tensors of heads with common strides, by their
// elements; otherwise the whole ranges are compared.
bool overlap(const Operand& a, const Operand& b);

// Null, alignment and overlap checks of a call's operands: no written operand
// may overlap another one, unless `alias` names the pair (written, read) that
// may be the very same tensor.
muon_status check_operands(const std::vector<Operand>& ops, std::string* detail, int alias_written = -1,
                           int alias_read_a = -1, int alias_read_b = -1);

// The same with any number of pairs (written, read) that may be one tensor.
typedef std::pair<int, int> Alias;
muon_status check_operands(const std::vector<Operand>& ops, std::string* detail, const std::vector<Alias>& same);

// A tensor [batch, tokens, heads, dim] of `size`-byte elements: its dimensions
// nest, and its offsets stay far inside 64 bits.  `op` receives it as runs of
// one pitch: the outer dimensions that follow one another, and in each run all
// that lies within.
muon_status head_operand(const char* name, const void* p, const muon_head_strides* s, int64_t batch, int64_t tokens,
                         int64_t heads, int64_t dim, int size, bool written, Operand* op, std::string* detail);

// Sizes and scalars of a call on query and key heads.
muon_status check_heads(muon_dtype dt, muon_dtype param_dt, int64_t batch, int64_t tokens, int32_t heads_q,
                        int32_t heads_k, bool keys, int32_t dim, float eps, const float* cos, const float* sin,
                        int64_t table_rows, int32_t rot, int32_t interleaved, const int64_t* positions,
                        int64_t positions_batch, std::string* detail);

muon_status check_logp(int64_t tokens, int64_t vocab, const std::vector<int64_t>& pitches, muon_dtype dt, float scale,
                       std::string* detail);
muon_status check_policy(int64_t tokens, float clip_low, float clip_high, float beta, std::string* detail);
muon_status check_preference(int64_t tokens, int64_t pairs, float beta, float margin, float smoothing,
                             int32_t average, std::string* detail);

muon_status check_op_dtype(muon_dtype dt, const char* what, std::string* detail);

// rows >= 0, cols in 1 .. max_cols, every pitch (elements) >= cols, and sizes
// whose offsets stay far inside 64 bits.
muon_status check_rows(int64_t rows, int64_t cols, int64_t max_cols, const std::vector<int64_t>& pitches,
                       std::string* detail);

// 0 <= p <= 1; a row counter of 32 bits.
muon_status check_dropout(float p, int64_t rows, const uint64_t* offset_dev, std::string* detail);

muon_status check_op_workspace(const void* workspace, size_t bytes, size_t need, std::string* detail);

// Bytes of the backward pass's partial sums (none for few rows).
inline size_t norm_workspace_bytes(int64_t rows, int64_t cols) {
  return size_t(norm_bwd_split(rows, cols).parts) * 2 * size_t(cols) * 4;
}
// The loss's terms (a double for each 16 experts), a counter of 16 bytes, and
// per workgroup: experts floats, experts counts, one count.  None for a lone
// workgroup.
constexpr int64_t kRouteTerms = kRouteMaxExperts / 16;
inline size_t route_workspace_bytes(int64_t rows, int64_t experts) {
  const int64_t parts = route_parts(rows, experts);
  return parts > 1 ? size_t(kRouteTerms) * 8 + 16 + size_t(parts) * (size_t(experts) * 8 + 4) : 0;
}

// Partial sums of dgamma: none where one workgroup takes all rows of a kind.
inline size_t heads_workspace_bytes(int64_t rows_q, int64_t rows_k, int64_t dim) {
  const HeadSplit s = head_split(rows_q, rows_k);
  return size_t((s.q > 1 ? s.q : 0) + (s.k > 1 ? s.k : 0)) * size_t(dim) * 4;
}
inline size_t logp_workspace_bytes(int64_t tokens, int64_t vocab) {
  const int parts = logp_parts(tokens, vocab);
  return parts > 1 ? size_t(tokens) * size_t(parts) * 8 : 0;
}
inline size_t policy_workspace_bytes(int64_t tokens) {
  const int parts = policy_parts(tokens);
  return parts > 1 ? size_t(parts) * 24 : 0;
}
inline size_t preference_workspace_bytes(int64_t tokens, int64_t pairs) {
  return pref_lone(tokens, pairs) ? 0 : (size_t(2 * pairs) << pref_shift(tokens, pairs)) * 16;
}

// Sizes of a router call.
muon_status check_route(int64_t tokens, int64_t ld, int32_t experts, int32_t k, int32_t renorm, float coef,
                        muon_dtype dt, std::string* detail);

}  // namespace muon
