// C ABI entry points of the training operators (include/muon.h): layer norm,
// dropout, the two fused, and the expert router.  Validation, then kernels on
// the caller's stream; nothing is allocated, kept or waited for.
#include <hip/hip_runtime.h>

#include <cmath>
#include <string>
#include <vector>

#include "api_ops.hpp"

namespace {

using namespace muon::api;
using muon::Operand;

muon::DropArgs drop_args(float p, uint64_t seed, uint64_t offset, const uint64_t* offset_dev) {
  muon::DropArgs d{};
  d.thresh = uint32_t(std::rint(double(p) * 65536.0));
  d.scale = d.thresh < 65536 ? float(65536.0 / double(65536 - d.thresh)) : 0.0f;
  d.k0 = uint32_t(seed);
  d.k1 = uint32_t(seed >> 32);
  d.offset = offset;
  d.offset_dev = offset_dev;
  return d;
}

muon_status norm_fwd(const void* x, int64_t ld_x, const void* res, int64_t ld_res, muon_dtype dt, const void* gamma,
                     const void* beta, muon_dtype param_dt, int64_t rows, int64_t cols, float eps,
                     const muon::DropArgs* drop, void* h, int64_t ld_h, void* y, int64_t ld_y, float* mean,
                     float* rstd, void* stream, std::string* d) {
  MUON_TRY(muon::check_op_dtype(dt, "dt", d));
  MUON_TRY(muon::check_op_dtype(param_dt, "param_dt", d));
  std::vector<int64_t> lds{ld_x, ld_y};
  if (drop) lds.insert(lds.end(), {ld_res, ld_h});
  MUON_TRY(muon::check_rows(rows, cols, muon::kNormMaxCols, lds, d));
  if (!(std::isfinite(eps) && eps > 0.0f)) {
    *d = "eps must be finite and > 0";
    return MUON_ERR_INVALID_ARG;
  }
  std::vector<Operand> ops{matrix("x", x, rows, cols, ld_x, dt, false),
                           matrix("y", y, rows, cols, ld_y, dt, true),
                           vec("gamma", gamma, cols, elem(param_dt), false, true),
                           vec("beta", beta, cols, elem(param_dt), false, true),
                           vec("mean", mean, rows, 4, true, true),
                           vec("rstd", rstd, rows, 4, true, true)};
  if (drop) {
    ops.push_back(matrix("residual", res, rows, cols, ld_res, dt, false));
    ops.push_back(matrix("h", h, rows, cols, ld_h, dt, true));
    ops.push_back(vec("offset_dev", drop->offset_dev, 1, 8, false, true));
  }
  MUON_TRY(muon::check_operands(ops, d, 7, 6));  // h may be the residual itself
  if (rows == 0) return MUON_OK;
  muon::NormFwdArgs a{};
  a.x = x; a.res = res; a.h = h; a.y = y; a.gamma = gamma; a.beta = beta; a.mean = mean; a.rstd = rstd;
  a.rows = rows; a.ld_x = ld_x; a.ld_res = ld_res; a.ld_h = ld_h; a.ld_y = ld_y;
  a.cols = int(cols);
  a.eps = eps;
  if (drop) a.drop = *drop;
  return launched(muon::run_norm_fwd(a, dt == MUON_BF16, param_dt == MUON_BF16, drop != nullptr, (hipStream_t)stream));
}

muon_status norm_bwd(const void* dy, int64_t ld_dy, const void* dh, int64_t ld_dh, const void* x, int64_t ld_x,
                     muon_dtype dt, const void* gamma, muon_dtype param_dt, const float* mean, const float* rstd,
                     int64_t rows, int64_t cols, const muon::DropArgs* drop, void* dx, int64_t ld_dx, void* dres,
                     int64_t ld_dres, void* dgamma, void* dbeta, void* workspace, size_t workspace_bytes,
                     void* stream, std::string* d) {
  MUON_TRY(muon::check_op_dtype(dt, "dt", d));
  MUON_TRY(muon::check_op_dtype(param_dt, "param_dt", d));
  std::vector<int64_t> lds{ld_dy, ld_x, ld_dx};
  if (drop) lds.push_back(ld_dres);
  if (drop && dh) lds.push_back(ld_dh);
  MUON_TRY(muon::check_rows(rows, cols, muon::kNormMaxCols, lds, d));
  const size_t need = (dgamma || dbeta) ? muon::norm_workspace_bytes(rows, cols) : 0;
  MUON_TRY(muon::check_op_workspace(workspace, workspace_bytes, need, d));
  std::vector<Operand> ops{matrix("dy", dy, rows, cols, ld_dy, dt, false),
                           matrix(drop ? "h" : "x", x, rows, cols, ld_x, dt, false),
                           matrix("dx", dx, rows, cols, ld_dx, dt, true),
                           vec("gamma", gamma, cols, elem(param_dt), false, true),
                           vec("mean", mean, rows, 4, false),
                           vec("rstd", rstd, rows, 4, false),
                           vec("dgamma", dgamma, cols, elem(param_dt), true, true),
                           vec("dbeta", dbeta, cols, elem(param_dt), true, true),
                           vec("workspace", need ? workspace : nullptr, int64_t(need / 4), 4, true, true)};
  if (drop) {
    ops.push_back(matrix("dresidual", dres, rows, cols, ld_dres, dt, true));
    ops.push_back(matrix("dh", dh, rows, cols, ld_dh, dt, false, true));
    ops.push_back(vec("offset_dev", drop->offset_dev, 1, 8, false, true));
  }
  MUON_TRY(muon::check_operands(ops, d));
  if (rows == 0 && !dgamma && !dbeta) return MUON_OK;  // with no row the gradients of gamma and beta are 0
  muon::NormBwdArgs a{};
  a.dy = dy; a.x = x; a.dh = drop ? dh : nullptr; a.gamma = gamma; a.mean = mean; a.rstd = rstd;
  a.dx = dx; a.dres = dres; a.dgamma = dgamma; a.dbeta = dbeta; a.part = (float*)workspace;
  a.parts = muon::norm_bwd_split(rows, cols).parts;
  a.rows = rows; a.ld_dy = ld_dy; a.ld_x = ld_x; a.ld_dh = ld_dh; a.ld_dx = ld_dx; a.ld_dres = ld_dres;
  a.cols = int(cols);
  if (drop) a.drop = *drop;
  return launched(muon::run_norm_bwd(a, dt == MUON_BF16, param_dt == MUON_BF16, drop != nullptr, (hipStream_t)stream));
}

}  // namespace

extern "C" {

muon_status muon_layer_norm_workspace_bytes(int64_t rows, int64_t cols, size_t* bytes) {
  return guarded([&](std::string* d) {
    if (!bytes) {
      *d = "null output pointer";
      return MUON_ERR_INVALID_ARG;
    }
    MUON_TRY(muon::check_rows(rows, cols, muon::kNormMaxCols, {}, d));
    *bytes = muon::norm_workspace_bytes(rows, cols);
    return MUON_OK;
  });
}

muon_status muon_layer_norm_fwd(const void* x, int64_t ld_x, muon_dtype dt, const void* gamma, const void* beta,
                                muon_dtype param_dt, int64_t rows, int64_t cols, float eps, void* y, int64_t ld_y,
                                float* mean, float* rstd, void* stream) {
  return guarded([&](std::string* d) {
    return norm_fwd(x, ld_x, nullptr, 0, dt, gamma, beta, param_dt, rows, cols, eps, nullptr, nullptr, 0, y, ld_y,
                    mean, rstd, stream, d);
  });
}

muon_status muon_layer_norm_bwd(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, muon_dtype dt,
                                const void* gamma, muon_dtype param_dt, const float* mean, const float* rstd,
                                int64_t rows, int64_t cols, void* dx, int64_t ld_dx, void* dgamma, void* dbeta,
                                void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&](std::string* d) {
    return norm_bwd(dy, ld_dy, nullptr, 0, x, ld_x, dt, gamma, param_dt, mean, rstd, rows, cols, nullptr, dx, ld_dx,
                    nullptr, 0, dgamma, dbeta, workspace, workspace_bytes, stream, d);
  });
}

muon_status muon_dropout(const void* x, int64_t ld_x, const void* residual, int64_t ld_res, muon_dtype dt,
                         int64_t rows, int64_t cols, float p, uint64_t seed, uint64_t offset,
                         const uint64_t* offset_dev, void* out, int64_t ld_out, void* stream) {
  return guarded([&](std::string* d) {
    MUON_TRY(muon::check_op_dtype(dt, "dt", d));
    std::vector<int64_t> lds{ld_x, ld_out};
    if (residual) lds.push_back(ld_res);
    MUON_TRY(muon::check_rows(rows, cols, int64_t(1) << 34, lds, d));
    MUON_TRY(muon::check_dropout(p, rows, offset_dev, d));
    const std::vector<Operand> ops{matrix("out", out, rows, cols, ld_out, dt, true),
                                   matrix("x", x, rows, cols, ld_x, dt, false),
                                   matrix("residual", residual, rows, cols, ld_res, dt, false, true),
                                   vec("offset_dev", offset_dev, 1, 8, false, true)};
    MUON_TRY(muon::check_operands(ops, d, 0, 1, 2));  // out may be x or the residual itself
    if (rows == 0) return MUON_OK;
    muon::DropoutArgs a{};
    a.x = x; a.res = residual; a.out = out;
    a.rows = rows; a.cols = cols; a.ld_x = ld_x; a.ld_res = ld_res; a.ld_out = ld_out;
    a.drop = drop_args(p, seed, offset, offset_dev);
    return launched(muon::run_dropout(a, dt == MUON_BF16, (hipStream_t)stream));
  });
}

muon_status muon_dropout_add_layer_norm_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_res,
                                            muon_dtype dt, const void* gamma, const void* beta, muon_dtype param_dt,
                                            int64_t rows, int64_t cols, float eps, float p, uint64_t seed,
                                            uint64_t offset, const uint64_t* offset_dev, void* h, int64_t ld_h,
                                            void* y, int64_t ld_y, float* mean, float* rstd, void* stream) {
  return guarded([&](std::string* d) {
    MUON_TRY(muon::check_dropout(p, rows, offset_dev, d));
    const muon::DropArgs drop = drop_args(p, seed, offset, offset_dev);
    return norm_fwd(x, ld_x, residual, ld_res, dt, gamma, beta, param_dt, rows, cols, eps, &drop, h, ld_h, y, ld_y,
                    mean, rstd, stream, d);
  });
}

muon_status muon_dropout_add_layer_norm_bwd(const void* dy, int64_t ld_dy, const void* dh, int64_t ld_dh,
                                            const void* h, int64_t ld_h, muon_dtype dt, const void* gamma,
                                            muon_dtype param_dt, const float* mean, const float* rstd, int64_t rows,
                                            int64_t cols, float p, uint64_t seed, uint64_t offset,
                                            const uint64_t* offset_dev, void* dx, int64_t ld_dx, void* dresidual,
                                            int64_t ld_dres, void* dgamma, void* dbeta, void* workspace,
                                            size_t workspace_bytes, void* stream) {
  return guarded([&](std::string* d) {
    MUON_TRY(muon::check_dropout(p, rows, offset_dev, d));
    const muon::DropArgs drop = drop_args(p, seed, offset, offset_dev);
    return norm_bwd(dy, ld_dy, dh, ld_dh, h, ld_h, dt, gamma, param_dt, mean, rstd, rows, cols, &drop, dx, ld_dx,
                    dresidual, ld_dres, dgamma, dbeta, workspace, workspace_bytes, stream, d);
  });
}

muon_status muon_route_workspace_bytes(int64_t tokens, int32_t experts, size_t* bytes) {
  return guarded([&](std::string* d) {
    if (!bytes) {
      *d = "null output pointer";
      return MUON_ERR_INVALID_ARG;
    }
    MUON_TRY(muon::check_rows(tokens, experts, muon::kRouteMaxExperts, {}, d));
    *bytes = muon::route_workspace_bytes(tokens, experts);
    return MUON_OK;
  });
}

muon_status muon_route_fwd(const void* logits, int64_t ld, muon_dtype dt, int64_t tokens, int32_t experts, int32_t k,
                           const uint8_t* valid, int32_t renorm, float coef, int32_t* indices, float* gates,
                           int32_t* counts, int32_t* n_tokens, float* prob_mean, float* loss, void* workspace,
                           size_t workspace_bytes, void* stream) {
  return guarded([&](std::string* d) {
    MUON_TRY(muon::check_route(tokens, ld, experts, k, renorm, coef, dt, d));
    const size_t need = muon::route_workspace_bytes(tokens, experts);
    MUON_TRY(muon::check_op_workspace(workspace, workspace_bytes, need, d));
    const std::vector<Operand> ops{matrix("logits", logits, tokens, experts, ld, dt, false),
                                   vec("valid", valid, tokens, 1, false, true),
                                   vec("indices", indices, tokens * k, 4, true),
                                   vec("gates", gates, tokens * k, 4, true),
                                   vec("counts", counts, experts, 4, true),
                                   vec("n_tokens", n_tokens, 1, 4, true),
                                   vec("prob_mean", prob_mean, experts, 4, true, true),
                                   vec("loss", loss, 1, 4, true),
                                   vec("workspace", need ? workspace : nullptr, int64_t(need / 4), 4, true, true)};
    MUON_TRY(muon::check_operands(ops, d));
    muon::RouteArgs a{};
    a.logits = logits; a.valid = valid; a.rows = tokens; a.ld = ld; a.experts = experts; a.k = k;
    a.renorm = renorm; a.coef = coef; a.idx = indices; a.gates = gates; a.counts = counts; a.n_tokens = n_tokens;
    a.prob_mean = prob_mean; a.loss = loss;
    a.parts = int(muon::route_parts(tokens, experts));
    if (a.parts > 1) {
      a.terms = (double*)workspace;
      a.ticket = (uint32_t*)(a.terms + muon::kRouteTerms);
      a.part_p = (float*)(a.ticket + 4);
      a.part_c = (int32_t*)a.part_p + int64_t(a.parts) * experts;
      a.part_n = a.part_c + int64_t(a.parts) * experts;
    }
    return launched(muon::run_route_fwd(a, dt == MUON_BF16, (hipStream_t)stream));
  });
}

muon_status muon_route_bwd(const void* logits, int64_t ld, muon_dtype dt, int64_t tokens, int32_t experts, int32_t k,
                           const uint8_t* valid, int32_t renorm, float coef, const int32_t* indices,
                           const int32_t* counts, const int32_t* n_tokens, const float* dgates, const float* dloss,
                           void* dlogits, int64_t ld_d, void* stream) {
  return guarded([&](std::string* d) {
    MUON_TRY(muon::check_route(tokens, ld, experts, k, renorm, coef, dt, d));
    MUON_TRY(muon::check_rows(tokens, experts, muon::kRouteMaxExperts, {ld_d}, d));
    const std::vector<Operand> ops{matrix("logits", logits, tokens, experts, ld, dt, false),
                                   matrix("dlogits", dlogits, tokens, experts, ld_d, dt, true),
                                   vec("valid", valid, tokens, 1, false, true),
                                   vec("indices", indices, tokens * k, 4, false),
                                   vec("counts", counts, experts, 4, false),
                                   vec("n_tokens", n_tokens, 1, 4, false),
                                   vec("dgates", dgates, tokens * k, 4, false, true),
                                   vec("dloss", dloss, 1, 4, false, true)};
    MUON_TRY(muon::check_operands(ops, d));
    if (tokens == 0) return MUON_OK;
    muon::RouteBwdArgs a{};
    a.logits = logits; a.valid = valid; a.rows = tokens; a.ld = ld; a.ld_d = ld_d; a.experts = experts; a.k = k;
    a.renorm = renorm; a.coef = coef; a.idx = indices; a.counts = counts; a.n_tokens = n_tokens;
    a.dgates = dgates; a.dloss = dloss; a.dlogits = dlogits;
    return launched(muon::run_route_bwd(a, dt == MUON_BF16, (hipStream_t)stream));
  });
}

}  // extern "C"
