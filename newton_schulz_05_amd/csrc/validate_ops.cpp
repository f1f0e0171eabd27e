// Argument validation of the training operators (see validate_ops.hpp).
#include "validate_ops.hpp"

#include <cmath>

namespace muon {

namespace {

muon_status fail(muon_status s, std::string* detail, const std::string& d) {
  *detail = d;
  return s;
}

// Largest row count, pitch and element offset of an operand.
constexpr int64_t kMaxExtent = int64_t(1) << 40;

}  // namespace

bool overlap(const Operand& a, const Operand& b) {
  if (!a.p || !b.p || a.rows < 1 || b.rows < 1) return false;
  const uint64_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uint64_t a1 = a0 + uint64_t(a.rows - 1) * uint64_t(a.pitch) + uint64_t(a.width);
  const uint64_t b1 = b0 + uint64_t(b.rows - 1) * uint64_t(b.pitch) + uint64_t(b.width);
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.pitch != b.pitch || (a.rows == 1 && b.rows == 1)) return true;
  // runs of b lie d bytes after runs of a, modulo the pitch
  const uint64_t pitch = uint64_t(a.pitch);
  const uint64_t d = (b0 >= a0) ? (b0 - a0) % pitch : (pitch - (a0 - b0) % pitch) % pitch;
  return d < uint64_t(a.width) || d + uint64_t(b.width) > pitch;
}

muon_status check_operands(const std::vector<Operand>& ops, std::string* detail, int alias_written, int alias_read_a,
                           int alias_read_b) {
  for (const Operand& o : ops) {
    if (!o.p) {
      if (o.optional || o.rows < 1) continue;
      return fail(MUON_ERR_INVALID_ARG, detail, std::string(o.name) + " is null");
    }
    if (reinterpret_cast<uintptr_t>(o.p) % uintptr_t(o.align) != 0)
      return fail(MUON_ERR_ALIGNMENT, detail,
                  std::string(o.name) + " is not " + std::to_string(o.align) + "-byte aligned");
  }
  for (size_t i = 0; i < ops.size(); ++i) {
    if (!ops[i].written) continue;
    for (size_t j = 0; j < ops.size(); ++j) {
      if (j == i || (ops[j].written && j < i) || !overlap(ops[i], ops[j])) continue;
      if (int(i) == alias_written && (int(j) == alias_read_a || int(j) == alias_read_b) && ops[i].p == ops[j].p &&
          (ops[i].pitch == ops[j].pitch || ops[i].rows == 1))
        continue;
      return fail(MUON_ERR_INVALID_ARG, detail, std::string(ops[i].name) + " and " + ops[j].name + " overlap");
    }
  }
  return MUON_OK;
}

muon_status check_op_dtype(muon_dtype dt, const char* what, std::string* detail) {
  if (dt != MUON_F32 && dt != MUON_BF16)
    return fail(MUON_ERR_DTYPE, detail, std::string(what) + " must be MUON_F32 or MUON_BF16");
  return MUON_OK;
}

muon_status check_rows(int64_t rows, int64_t cols, int64_t max_cols, const std::vector<int64_t>& pitches,
                       std::string* detail) {
  if (rows < 0) return fail(MUON_ERR_SHAPE, detail, "rows must be >= 0");
  if (cols < 1 || cols > max_cols)
    return fail(MUON_ERR_SHAPE, detail, "cols must be in 1.." + std::to_string(max_cols));
  if (rows > kMaxExtent) return fail(MUON_ERR_SHAPE, detail, "too many rows");
  for (int64_t ld : pitches) {
    if (ld < cols) return fail(MUON_ERR_INVALID_ARG, detail, "a row stride is smaller than cols");
    if (ld > kMaxExtent || (rows > 1 && ld > kMaxExtent / rows))
      return fail(MUON_ERR_SHAPE, detail, "tensor too large");
  }
  return MUON_OK;
}

muon_status check_dropout(float p, int64_t rows, const uint64_t* offset_dev, std::string* detail) {
  if (!(p >= 0.0f && p <= 1.0f)) return fail(MUON_ERR_INVALID_ARG, detail, "p must be in [0, 1]");
  if (rows > int64_t(0xffffffff)) return fail(MUON_ERR_SHAPE, detail, "dropout counts rows in 32 bits");
  if (reinterpret_cast<uintptr_t>(offset_dev) % 8 != 0)
    return fail(MUON_ERR_ALIGNMENT, detail, "offset_dev is not 8-byte aligned");
  return MUON_OK;
}

muon_status check_op_workspace(const void* workspace, size_t bytes, size_t need, std::string* detail) {
  if (need == 0) return MUON_OK;
  if (!workspace) return fail(MUON_ERR_WORKSPACE, detail, "workspace is null");
  if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0)
    return fail(MUON_ERR_WORKSPACE, detail, "workspace is not 16-byte aligned");
  if (bytes < need)
    return fail(MUON_ERR_WORKSPACE, detail,
                "workspace has " + std::to_string(bytes) + " bytes, needs " + std::to_string(need));
  return MUON_OK;
}

muon_status check_route(int64_t tokens, int64_t ld, int32_t experts, int32_t k, int32_t renorm, float coef,
                        muon_dtype dt, std::string* detail) {
  muon_status s = check_op_dtype(dt, "dt", detail);
  if (s != MUON_OK) return s;
  if (experts < 1 || experts > kRouteMaxExperts)
    return fail(MUON_ERR_SHAPE, detail, "experts must be in 1.." + std::to_string(kRouteMaxExperts));
  if (k < 1 || k > kRouteMaxK || k > experts)
    return fail(MUON_ERR_SHAPE, detail, "k must be in 1..min(experts, " + std::to_string(kRouteMaxK) + ")");
  if ((s = check_rows(tokens, experts, kRouteMaxExperts, {ld}, detail)) != MUON_OK) return s;
  if (tokens > int64_t(0x7fffffff) / k)
    return fail(MUON_ERR_SHAPE, detail, "tokens * k must fit in 32 bits (the counts' type)");
  if (renorm != 0 && renorm != 1) return fail(MUON_ERR_INVALID_ARG, detail, "renorm must be 0 or 1");
  if (!std::isfinite(coef)) return fail(MUON_ERR_INVALID_ARG, detail, "coef must be finite");
  return MUON_OK;
}

}  // namespace muon
