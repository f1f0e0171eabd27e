// Argument validation of the training operators (see validate_ops.hpp).
#include "validate_ops.hpp"

#include <algorithm>
#include <cmath>

namespace muon {

namespace {

muon_status fail(muon_status s, std::string* detail, const std::string& d) {
  *detail = d;
  return s;
}

// Largest row count, pitch and element offset of an operand.
constexpr int64_t kMaxExtent = int64_t(1) << 40;

// Two tensors of heads with common strides, b's first byte `d` behind a's: whether
// an entry of one meets an entry of the other.  Dimensions outermost first; what
// lies within one is no longer than its stride, so that at most a few distances
// t = (b's index - a's) come into question at each.
struct HeadPair {
  int64_t na[3], nb[3], s[3], wa, wb;
  int64_t span(const int64_t (&n)[3], int64_t w, int from) const {
    for (int i = from; i < 3; ++i) w += (n[i] - 1) * s[i];
    return w;
  }
  bool meet(int level, int64_t d) const {
    if (level == 3) return d < wa && -d < wb;
    const int64_t sa = span(na, wa, level + 1), sb = span(nb, wb, level + 1);
    if (s[level] == 0) return meet(level + 1, d);
    auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y != 0 && x < 0); };
    // -sb < d + t s < sa
    const int64_t lo = std::max(floor_div(-sb - d, s[level]) + 1, 1 - na[level]);
    const int64_t hi = std::min(-floor_div(-(sa - d), s[level]) - 1, nb[level] - 1);
    for (int64_t t = lo; t <= hi; ++t)
      if (meet(level + 1, d + t * s[level])) return true;
    return false;
  }
};

// Fills `p` if a and b have common strides.
bool common_strides(const Operand& a, const Operand& b, HeadPair* p) {
  if (!a.inner || !b.inner) return false;
  struct Dim {
    int64_t na, nb, s;
  } d[3];
  for (int i = 0; i < 3; ++i) {
    if (a.n[i] > 1 && b.n[i] > 1 && a.s[i] != b.s[i]) return false;
    d[i] = {a.n[i], b.n[i], a.n[i] > 1 ? a.s[i] : b.n[i] > 1 ? b.s[i] : 0};
  }
  std::sort(d, d + 3, [](const Dim& x, const Dim& y) { return x.s > y.s; });
  for (int i = 0; i < 3; ++i) {
    p->na[i] = d[i].na;
    p->nb[i] = d[i].nb;
    p->s[i] = d[i].s;
  }
  p->wa = a.inner;
  p->wb = b.inner;
  // a dimension that one tensor has alone may be shorter than what the other has within it
  for (int i = 0; i < 3; ++i)
    if (p->s[i] > 0 && (p->span(p->na, p->wa, i + 1) > p->s[i] || p->span(p->nb, p->wb, i + 1) > p->s[i])) return false;
  return true;
}

}  // namespace

bool overlap(const Operand& a, const Operand& b) {
  if (!a.p || !b.p || a.rows < 1 || b.rows < 1) return false;
  const uint64_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uint64_t a1 = a0 + uint64_t(a.rows - 1) * uint64_t(a.pitch) + uint64_t(a.width);
  const uint64_t b1 = b0 + uint64_t(b.rows - 1) * uint64_t(b.pitch) + uint64_t(b.width);
  if (a1 <= b0 || b1 <= a0) return false;
  HeadPair h;
  if (common_strides(a, b, &h)) return h.meet(0, int64_t(b0 - a0));
  if (a.pitch != b.pitch || (a.rows == 1 && b.rows == 1)) return true;
  // runs of b lie d bytes after runs of a, modulo the pitch
  const uint64_t pitch = uint64_t(a.pitch);
  const uint64_t d = (b0 >= a0) ? (b0 - a0) % pitch : (pitch - (a0 - b0) % pitch) % pitch;
  return d < uint64_t(a.width) || d + uint64_t(b.width) > pitch;
}

muon_status check_operands(const std::vector<Operand>& ops, std::string* detail, int alias_written, int alias_read_a,
                           int alias_read_b) {
  return check_operands(ops, detail, {{alias_written, alias_read_a}, {alias_written, alias_read_b}});
}

muon_status check_operands(const std::vector<Operand>& ops, std::string* detail, const std::vector<Alias>& same) {
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
      const bool may = std::find(same.begin(), same.end(), Alias(int(i), int(j))) != same.end();
      if (may && ops[i].p == ops[j].p && (ops[i].pitch == ops[j].pitch || ops[i].rows == 1)) continue;
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

muon_status head_operand(const char* name, const void* p, const muon_head_strides* s, int64_t batch, int64_t tokens,
                         int64_t heads, int64_t dim, int size, bool written, Operand* op, std::string* detail) {
  *op = Operand{name, p, batch * tokens * heads > 0 ? 1 : 0, dim * size, dim * size, size, written, false};
  if (op->rows == 0) return MUON_OK;
  if (!s) return fail(MUON_ERR_INVALID_ARG, detail, std::string(name) + ": strides are null");
  struct Dim {
    int64_t n, stride;
  } d[3] = {{batch, s->batch}, {tokens, s->token}, {heads, s->head}};
  // innermost first; a dimension of one entry has no stride
  std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return (a.n > 1 ? a.stride : 0) < (b.n > 1 ? b.stride : 0); });
  int64_t span = dim;  // elements up to the end of the dimensions so far
  for (const Dim& x : d) {
    if (x.n == 1) continue;
    if (x.stride < span)
      return fail(MUON_ERR_INVALID_ARG, detail,
                  std::string(name) + ": the dimensions do not nest (a stride is smaller than what lies within)");
    if (x.stride > kMaxExtent / x.n) return fail(MUON_ERR_SHAPE, detail, std::string(name) + ": tensor too large");
    span += (x.n - 1) * x.stride;
  }
  op->inner = dim * size;
  const int64_t ns[3] = {batch, tokens, heads}, strides[3] = {s->batch, s->token, s->head};
  for (int i = 0; i < 3; ++i) {
    op->n[i] = ns[i];
    op->s[i] = ns[i] > 1 ? strides[i] * size : 0;
  }
  // outermost first: dimensions that follow one another without a gap are one
  op->width = span * size;
  op->pitch = span * size;
  for (int i = 2; i >= 0; --i) {
    if (d[i].n == 1) continue;
    if (op->rows > 1 && op->pitch != d[i].n * d[i].stride * size) break;
    op->rows *= d[i].n;
    op->pitch = d[i].stride * size;
    span -= (d[i].n - 1) * d[i].stride;
    op->width = span * size;
  }
  return MUON_OK;
}

muon_status check_heads(muon_dtype dt, muon_dtype param_dt, int64_t batch, int64_t tokens, int32_t heads_q,
                        int32_t heads_k, bool keys, int32_t dim, float eps, const float* cos, const float* sin,
                        int64_t table_rows, int32_t rot, int32_t interleaved, const int64_t* positions,
                        int64_t positions_batch, std::string* detail) {
  muon_status s = check_op_dtype(dt, "dt", detail);
  if (s == MUON_OK) s = check_op_dtype(param_dt, "param_dt", detail);
  if (s != MUON_OK) return s;
  if (dim < 1 || dim > kHeadMaxDim)
    return fail(MUON_ERR_SHAPE, detail, "dim must be in 1.." + std::to_string(kHeadMaxDim));
  if (batch < 0 || tokens < 0) return fail(MUON_ERR_SHAPE, detail, "batch and tokens must be >= 0");
  if (heads_q < 1) return fail(MUON_ERR_SHAPE, detail, "heads_q must be >= 1");
  if (keys ? heads_k < 1 : heads_k != 0)
    return fail(MUON_ERR_SHAPE, detail, "heads_k must be >= 1, or 0 without keys");
  const int64_t heads = std::max(heads_q, heads_k);
  if (batch > kHeadMaxRows || tokens > kHeadMaxRows || batch * tokens > kHeadMaxRows / heads)
    return fail(MUON_ERR_SHAPE, detail, "batch * tokens * heads must be below 2^31");
  if (!(std::isfinite(eps) && eps > 0.0f)) return fail(MUON_ERR_INVALID_ARG, detail, "eps must be finite and > 0");
  if (interleaved != 0 && interleaved != 1) return fail(MUON_ERR_INVALID_ARG, detail, "interleaved must be 0 or 1");
  if (rot < 0 || rot > dim || rot % 2 != 0)
    return fail(MUON_ERR_SHAPE, detail, "rot must be even and in 0..dim");
  if (rot > 0) {
    if (table_rows < 0 || table_rows > kMaxExtent / rot)
      return fail(MUON_ERR_SHAPE, detail, "table_rows is out of range");
    if (table_rows > 0 && (!cos || !sin)) return fail(MUON_ERR_INVALID_ARG, detail, "cos or sin is null");
    if (!positions && batch > 0 && table_rows < tokens)
      return fail(MUON_ERR_SHAPE, detail, "cos and sin have fewer rows than there are tokens");
    if (positions && batch > 1 && positions_batch != 0 && positions_batch < tokens)
      return fail(MUON_ERR_INVALID_ARG, detail, "positions_batch must be 0 or at least tokens");
    if (positions_batch < 0 || (batch > 1 && positions_batch > kMaxExtent / batch))
      return fail(MUON_ERR_SHAPE, detail, "positions_batch is out of range");
  }
  return MUON_OK;
}

muon_status check_logp(int64_t tokens, int64_t vocab, const std::vector<int64_t>& pitches, muon_dtype dt, float scale,
                       std::string* detail) {
  muon_status s = check_op_dtype(dt, "dt", detail);
  if (s == MUON_OK) s = check_rows(tokens, vocab, kLogpMaxVocab, pitches, detail);
  if (s != MUON_OK) return s;
  if (tokens > kHeadMaxRows) return fail(MUON_ERR_SHAPE, detail, "tokens must be below 2^31");
  // the factor under the exponential is scale log2(e)
  if (!(scale > 0.0f && scale <= 1e30f)) return fail(MUON_ERR_INVALID_ARG, detail, "scale must be > 0 and at most 1e30");
  return MUON_OK;
}

muon_status check_policy(int64_t tokens, float clip_low, float clip_high, float beta, std::string* detail) {
  if (tokens < 0 || tokens > kLossMaxTokens) return fail(MUON_ERR_SHAPE, detail, "tokens is out of range");
  if (!(clip_low >= 0.0f && clip_low <= 1.0f)) return fail(MUON_ERR_INVALID_ARG, detail, "clip_low must be in [0, 1]");
  if (!(std::isfinite(clip_high) && clip_high >= 0.0f))
    return fail(MUON_ERR_INVALID_ARG, detail, "clip_high must be finite and >= 0");
  if (!std::isfinite(beta)) return fail(MUON_ERR_INVALID_ARG, detail, "beta must be finite");
  return MUON_OK;
}

muon_status check_preference(int64_t tokens, int64_t pairs, float beta, float margin, float smoothing,
                             int32_t average, std::string* detail) {
  if (tokens < 0 || tokens > kLossMaxTokens) return fail(MUON_ERR_SHAPE, detail, "tokens is out of range");
  if (pairs < 0 || pairs > kPrefMaxPairs)
    return fail(MUON_ERR_SHAPE, detail, "pairs must be in 0.." + std::to_string(kPrefMaxPairs));
  if (!std::isfinite(beta) || !std::isfinite(margin))
    return fail(MUON_ERR_INVALID_ARG, detail, "beta and margin must be finite");
  if (!(smoothing >= 0.0f && smoothing <= 1.0f))
    return fail(MUON_ERR_INVALID_ARG, detail, "smoothing must be in [0, 1]");
  if (average != 0 && average != 1) return fail(MUON_ERR_INVALID_ARG, detail, "average must be 0 or 1");
  return MUON_OK;
}

}  // namespace muon
