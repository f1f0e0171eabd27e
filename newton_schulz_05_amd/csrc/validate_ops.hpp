// Argument validation of the training operators' entry points (layer norm,
// dropout, router).  Pure C++ (no HIP calls), like validate.hpp: each function
// returns MUON_OK, or an error status with `detail` filled, before anything is
// enqueued, and none of them touches device memory.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <string>
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
};

// Whether two operands share a byte.  Runs of one common pitch are compared
// by their place within the pitch, so that column slices of one buffer count
// as apart; otherwise the whole ranges are compared.
bool overlap(const Operand& a, const Operand& b);

// Null, alignment and overlap checks of a call's operands: no written operand
// may overlap another one, unless `alias` names the pair (written, read) that
// may be the very same tensor.
muon_status check_operands(const std::vector<Operand>& ops, std::string* detail, int alias_written = -1,
                           int alias_read_a = -1, int alias_read_b = -1);

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

// Sizes of a router call.
muon_status check_route(int64_t tokens, int64_t ld, int32_t experts, int32_t k, int32_t renorm, float coef,
                        muon_dtype dt, std::string* detail);

}  // namespace muon
