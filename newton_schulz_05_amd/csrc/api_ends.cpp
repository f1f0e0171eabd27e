// C ABI entry points of the operators at the two ends of a training step
// (include/muon.h): the norm and rotation of query and key heads, token
// log-probabilities, the policy loss and the preference loss.  Validation, then
// kernels on the caller's stream; nothing is allocated, kept or waited for.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <utility>
#include <vector>

#include "api_ops.hpp"

namespace {

using namespace muon::api;
using muon::Operand;

// What a call on heads is given, queries and keys alike.
struct HeadCall {
  muon_dtype dt, param_dt;
  int64_t batch, tokens;
  int32_t heads_q, heads_k, dim;
  float eps;
  const float *cos, *sin;
  int64_t table_rows;
  int32_t rot, interleaved;
  const int64_t* positions;
  int64_t positions_batch;
};
struct HeadTensors {
  const char *x_name, *dy_name, *out_name, *gamma_name, *dgamma_name;
  const void* x;
  const muon_head_strides* s_x;
  const void* dy;  // backward
  const muon_head_strides* s_dy;
  void* out;
  const muon_head_strides* s_out;
  const void* gamma;
  void* dgamma;
  int32_t heads;
};

// The same elements at the same places: strides of dimensions of one entry do
// not count.
bool same_strides(const HeadCall& c, int32_t heads, const muon_head_strides* a, const muon_head_strides* b) {
  return a && b && (c.batch <= 1 || a->batch == b->batch) && (c.tokens <= 1 || a->token == b->token) &&
         (heads <= 1 || a->head == b->head);
}

// Adds the operands of one kind of heads; the pair (out, what it may be itself)
// to `same`.
muon_status add_operands(const HeadCall& c, const HeadTensors& h, bool backward, std::vector<Operand>* ops,
                         std::vector<muon::Alias>* same, std::string* d) {
  const int size = int(elem(c.dt));
  Operand o;
  const int x = int(ops->size());
  MUON_TRY(muon::head_operand(h.x_name, h.x, h.s_x, c.batch, c.tokens, h.heads, c.dim, size, false, &o, d));
  ops->push_back(o);
  if (backward) {
    MUON_TRY(muon::head_operand(h.dy_name, h.dy, h.s_dy, c.batch, c.tokens, h.heads, c.dim, size, false, &o, d));
    ops->push_back(o);
  }
  MUON_TRY(muon::head_operand(h.out_name, h.out, h.s_out, c.batch, c.tokens, h.heads, c.dim, size, true, &o, d));
  ops->push_back(o);
  const int out = int(ops->size()) - 1, twin = backward ? x + 1 : x;
  if (same_strides(c, h.heads, h.s_out, backward ? h.s_dy : h.s_x)) same->push_back({out, twin});
  ops->push_back(vec(h.gamma_name, h.gamma, c.dim, elem(c.param_dt), false, true));
  if (backward) ops->push_back(vec(h.dgamma_name, h.dgamma, c.dim, elem(c.param_dt), true, true));
  return MUON_OK;
}

// Rows in the order of x's memory: the dimension of the smallest stride first.
muon::HeadRows head_rows(const HeadCall& c, const HeadTensors& h) {
  muon::HeadRows r{};
  r.x = h.x; r.dy = h.dy; r.out = h.out; r.gamma = h.gamma; r.dgamma = h.dgamma;
  r.rows = uint32_t(c.batch * c.tokens * h.heads);
  r.n0 = r.n1 = muon::fast_div(1);
  if (r.rows == 0) return r;
  struct Dim {
    int64_t n, x, dy, out, pos;
  } d[3] = {{c.batch, h.s_x->batch, h.s_dy ? h.s_dy->batch : 0, h.s_out->batch, c.positions ? c.positions_batch : 0},
            {c.tokens, h.s_x->token, h.s_dy ? h.s_dy->token : 0, h.s_out->token, 1},
            {h.heads, h.s_x->head, h.s_dy ? h.s_dy->head : 0, h.s_out->head, 0}};
  std::stable_sort(d, d + 3, [](const Dim& a, const Dim& b) { return (a.n > 1 ? a.x : 0) < (b.n > 1 ? b.x : 0); });
  r.n0 = muon::fast_div(d[0].n);
  r.n1 = muon::fast_div(d[1].n);
  for (int i = 0; i < 3; ++i) {
    r.s_x[i] = d[i].x;
    r.s_dy[i] = d[i].dy;
    r.s_out[i] = d[i].out;
    r.s_pos[i] = d[i].pos;
  }
  return r;
}

muon_status heads(const HeadCall& c, const HeadTensors& q, const HeadTensors& k, bool backward, void* workspace,
                  size_t workspace_bytes, void* stream, std::string* d) {
  const bool keys = k.heads != 0 || k.x || k.out || k.dy;
  MUON_TRY(muon::check_heads(c.dt, c.param_dt, c.batch, c.tokens, c.heads_q, c.heads_k, keys, c.dim, c.eps, c.cos, c.sin,
                             c.table_rows, c.rot, c.interleaved, c.positions, c.positions_batch, d));
  if (!keys && k.dgamma) {
    *d = "dgamma_k is given without keys";
    return MUON_ERR_INVALID_ARG;
  }
  const int64_t rows_q = c.batch * c.tokens * c.heads_q, rows_k = c.batch * c.tokens * c.heads_k;
  const size_t need = q.dgamma || k.dgamma ? muon::heads_workspace_bytes(rows_q, rows_k, c.dim) : 0;
  MUON_TRY(muon::check_op_workspace(workspace, workspace_bytes, need, d));
  std::vector<Operand> ops;
  std::vector<muon::Alias> same;
  MUON_TRY(add_operands(c, q, backward, &ops, &same, d));
  if (keys) MUON_TRY(add_operands(c, k, backward, &ops, &same, d));
  if (c.rot > 0) {
    ops.push_back(vec("cos", c.cos, c.table_rows * (c.rot / 2), 4, false));
    ops.push_back(vec("sin", c.sin, c.table_rows * (c.rot / 2), 4, false));
    const int64_t words = rows_q > 0 ? (c.batch - 1) * c.positions_batch + c.tokens : 0;
    ops.push_back(vec("positions", c.positions, words, 8, false, true));
  }
  if (need) ops.push_back(vec("workspace", workspace, int64_t(need / 4), 4, true));
  MUON_TRY(muon::check_operands(ops, d, same));
  if (rows_q == 0 && !q.dgamma && !k.dgamma) return MUON_OK;  // with no row the gradients of gamma are 0
  muon::HeadArgs a{};
  a.q = head_rows(c, q);
  a.k = head_rows(c, k);
  a.cos = c.cos; a.sin = c.sin; a.positions = c.rot > 0 ? c.positions : nullptr; a.table_rows = c.table_rows;
  a.dim = c.dim; a.rot = c.rot; a.eps = c.eps; a.wbf16 = c.param_dt == MUON_BF16;
  const bool bf16 = c.dt == MUON_BF16;
  if (!backward) return launched(muon::run_heads_fwd(a, bf16, c.interleaved != 0, (hipStream_t)stream));
  const muon::HeadSplit s = muon::head_split(rows_q, rows_k);
  a.q.wgs = s.q;
  a.k.wgs = s.k;
  float* part = (float*)workspace;
  if (q.dgamma && s.q > 1) a.q.part = part;
  if (k.dgamma && s.k > 1) a.k.part = part + (s.q > 1 ? int64_t(s.q) * c.dim : 0);
  return launched(muon::run_heads_bwd(a, bf16, c.interleaved != 0, (hipStream_t)stream));
}

template <typename F> muon_status bytes_of(size_t* bytes, F f) {
  return guarded([&](std::string* d) {
    if (!bytes) {
      *d = "null output pointer";
      return MUON_ERR_INVALID_ARG;
    }
    return f(d);
  });
}

}  // namespace

extern "C" {

muon_status muon_qk_norm_rope_fwd(const void* q, const muon_head_strides* s_q, const void* k,
                                  const muon_head_strides* s_k, muon_dtype dt, int64_t batch, int64_t tokens,
                                  int32_t heads_q, int32_t heads_k, int32_t dim, const void* gamma_q,
                                  const void* gamma_k, muon_dtype param_dt, float eps, const float* cos,
                                  const float* sin, int64_t table_rows, int32_t rot, int32_t interleaved,
                                  const int64_t* positions, int64_t positions_batch, void* q_out,
                                  const muon_head_strides* s_qo, void* k_out, const muon_head_strides* s_ko,
                                  void* stream) {
  return guarded([&](std::string* d) {
    const HeadCall c{dt, param_dt, batch, tokens, heads_q, heads_k, dim, eps, cos, sin, table_rows, rot, interleaved,
                     positions, positions_batch};
    const HeadTensors tq{"q", "", "q_out", "gamma_q", "", q, s_q, nullptr, nullptr, q_out, s_qo, gamma_q, nullptr,
                         heads_q};
    const HeadTensors tk{"k", "", "k_out", "gamma_k", "", k, s_k, nullptr, nullptr, k_out, s_ko, gamma_k, nullptr,
                         heads_k};
    return heads(c, tq, tk, false, nullptr, 0, stream, d);
  });
}

muon_status muon_qk_norm_rope_workspace_bytes(int64_t rows_q, int64_t rows_k, int32_t dim, size_t* bytes) {
  return bytes_of(bytes, [&](std::string* d) {
    if (dim < 1 || dim > muon::kHeadMaxDim || rows_q < 0 || rows_k < 0 || rows_q > muon::kHeadMaxRows ||
        rows_k > muon::kHeadMaxRows) {
      *d = "rows or dim out of range";
      return MUON_ERR_SHAPE;
    }
    *bytes = muon::heads_workspace_bytes(rows_q, rows_k, dim);
    return MUON_OK;
  });
}

muon_status muon_qk_norm_rope_bwd(const void* dq_out, const muon_head_strides* s_dqo, const void* dk_out,
                                  const muon_head_strides* s_dko, const void* q, const muon_head_strides* s_q,
                                  const void* k, const muon_head_strides* s_k, muon_dtype dt, int64_t batch,
                                  int64_t tokens, int32_t heads_q, int32_t heads_k, int32_t dim,
                                  const void* gamma_q, const void* gamma_k, muon_dtype param_dt, float eps,
                                  const float* cos, const float* sin, int64_t table_rows, int32_t rot,
                                  int32_t interleaved, const int64_t* positions, int64_t positions_batch, void* dq,
                                  const muon_head_strides* s_dq, void* dk, const muon_head_strides* s_dk,
                                  void* dgamma_q, void* dgamma_k, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  return guarded([&](std::string* d) {
    const HeadCall c{dt, param_dt, batch, tokens, heads_q, heads_k, dim, eps, cos, sin, table_rows, rot, interleaved,
                     positions, positions_batch};
    const HeadTensors tq{"q", "dq_out", "dq", "gamma_q", "dgamma_q", q, s_q, dq_out, s_dqo, dq, s_dq, gamma_q, dgamma_q,
                         heads_q};
    const HeadTensors tk{"k", "dk_out", "dk", "gamma_k", "dgamma_k", k, s_k, dk_out, s_dko, dk, s_dk, gamma_k, dgamma_k,
                         heads_k};
    return heads(c, tq, tk, true, workspace, workspace_bytes, stream, d);
  });
}

muon_status muon_token_logp_workspace_bytes(int64_t tokens, int64_t vocab, size_t* bytes) {
  return bytes_of(bytes, [&](std::string* d) {
    MUON_TRY(muon::check_logp(tokens, vocab, {}, MUON_F32, 1.0f, d));
    *bytes = muon::logp_workspace_bytes(tokens, vocab);
    return MUON_OK;
  });
}

muon_status muon_token_logp_fwd(const void* logits, int64_t ld, muon_dtype dt, int64_t tokens, int64_t vocab,
                                const int64_t* targets, float scale, float* logp, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return guarded([&](std::string* d) {
    MUON_TRY(muon::check_logp(tokens, vocab, {ld}, dt, scale, d));
    const size_t need = muon::logp_workspace_bytes(tokens, vocab);
    MUON_TRY(muon::check_op_workspace(workspace, workspace_bytes, need, d));
    std::vector<Operand> ops{matrix("logits", logits, tokens, vocab, ld, dt, false),
                             vec("targets", targets, tokens, 8, false),
                             vec("logp", logp, tokens, 4, true),
                             vec("lse", lse, tokens, 4, true)};
    if (need) ops.push_back(vec("workspace", workspace, int64_t(need / 4), 4, true));
    MUON_TRY(muon::check_operands(ops, d));
    muon::LogpArgs a{};
    a.logits = logits; a.targets = targets; a.rows = tokens; a.cols = vocab; a.ld = ld;
    a.scale = scale;
    a.scale2 = float(double(scale) * 1.4426950408889634);
    a.logp = logp; a.lse = lse;
    a.parts = muon::logp_parts(tokens, vocab);
    a.part = (float*)workspace;
    return launched(muon::run_logp_fwd(a, dt == MUON_BF16, (hipStream_t)stream));
  });
}

muon_status muon_token_logp_bwd(const void* logits, int64_t ld, muon_dtype dt, int64_t tokens, int64_t vocab,
                                const int64_t* targets, float scale, const float* logp, const float* lse,
                                const float* dlogp, void* dlogits, int64_t ld_d, void* stream) {
  return guarded([&](std::string* d) {
    MUON_TRY(muon::check_logp(tokens, vocab, {ld, ld_d}, dt, scale, d));
    const std::vector<Operand> ops{matrix("dlogits", dlogits, tokens, vocab, ld_d, dt, true),
                                   matrix("logits", logits, tokens, vocab, ld, dt, false),
                                   vec("targets", targets, tokens, 8, false),
                                   vec("logp", logp, tokens, 4, false),
                                   vec("lse", lse, tokens, 4, false),
                                   vec("dlogp", dlogp, tokens, 4, false)};
    MUON_TRY(muon::check_operands(ops, d, 0, 1));  // dlogits may be the logits themselves
    if (tokens == 0) return MUON_OK;
    muon::LogpBwdArgs a{};
    a.logits = logits; a.targets = targets; a.rows = tokens; a.cols = vocab; a.ld = ld; a.ld_d = ld_d;
    a.scale = scale;
    a.scale2 = float(double(scale) * 1.4426950408889634);
    a.logp = logp; a.lse = lse; a.dlogp = dlogp; a.dlogits = dlogits;
    return launched(muon::run_logp_bwd(a, dt == MUON_BF16, (hipStream_t)stream));
  });
}

muon_status muon_policy_loss_workspace_bytes(int64_t tokens, size_t* bytes) {
  return bytes_of(bytes, [&](std::string* d) {
    MUON_TRY(muon::check_policy(tokens, 0.0f, 0.0f, 0.0f, d));
    *bytes = muon::policy_workspace_bytes(tokens);
    return MUON_OK;
  });
}

muon_status muon_policy_loss(const float* logp, const float* old_logp, const float* ref_logp,
                             const float* advantages, const float* weight, int64_t tokens, float clip_low,
                             float clip_high, float beta, const float* dloss, float* loss, float* terms,
                             float* dlogp, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&](std::string* d) {
    MUON_TRY(muon::check_policy(tokens, clip_low, clip_high, beta, d));
    const size_t need = muon::policy_workspace_bytes(tokens);
    MUON_TRY(muon::check_op_workspace(workspace, workspace_bytes, need, d));
    std::vector<Operand> ops{vec("logp", logp, tokens, 4, false),
                             vec("old_logp", old_logp, tokens, 4, false, true),
                             vec("ref_logp", ref_logp, tokens, 4, false, true),
                             vec("advantages", advantages, tokens, 4, false),
                             vec("weight", weight, tokens, 4, false, true),
                             vec("dloss", dloss, 1, 4, false, true),
                             vec("loss", loss, 1, 4, true),
                             vec("terms", terms, 3, 4, true, true),
                             vec("dlogp", dlogp, tokens, 4, true, true)};
    if (need) ops.push_back(vec("workspace", workspace, int64_t(need / 8), 8, true));
    MUON_TRY(muon::check_operands(ops, d));
    muon::PolicyArgs a{};
    a.logp = logp; a.old_logp = old_logp; a.ref = ref_logp; a.adv = advantages; a.weight = weight; a.dloss = dloss;
    a.tokens = tokens;
    a.low = 1.0 - double(clip_low);
    a.high = 1.0 + double(clip_high);
    a.log_low = std::log(a.low);
    a.log_high = std::log(a.high);
    a.beta = beta;
    a.loss = loss; a.terms = terms; a.dlogp = dlogp;
    a.parts = muon::policy_parts(tokens);
    a.part = (double*)workspace;
    return launched(muon::run_policy_loss(a, (hipStream_t)stream));
  });
}

muon_status muon_preference_loss_workspace_bytes(int64_t tokens, int64_t pairs, size_t* bytes) {
  return bytes_of(bytes, [&](std::string* d) {
    MUON_TRY(muon::check_preference(tokens, pairs, 0.0f, 0.0f, 0.0f, 0, d));
    *bytes = muon::preference_workspace_bytes(tokens, pairs);
    return MUON_OK;
  });
}

muon_status muon_preference_loss(const float* logp, const float* ref_logp, const uint8_t* valid, int64_t tokens,
                                 const int64_t* offsets, int64_t pairs, const float* weight, float beta,
                                 float margin, float smoothing, int32_t average, const float* dloss, float* loss,
                                 float* rewards, float* dlogp, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  return guarded([&](std::string* d) {
    MUON_TRY(muon::check_preference(tokens, pairs, beta, margin, smoothing, average, d));
    const size_t need = muon::preference_workspace_bytes(tokens, pairs);
    MUON_TRY(muon::check_op_workspace(workspace, workspace_bytes, need, d));
    std::vector<Operand> ops{vec("logp", logp, tokens, 4, false),
                             vec("ref_logp", ref_logp, tokens, 4, false, true),
                             vec("valid", valid, tokens, 1, false, true),
                             vec("offsets", offsets, pairs > 0 ? 2 * pairs + 1 : 0, 8, false),
                             vec("weight", weight, pairs, 4, false, true),
                             vec("dloss", dloss, 1, 4, false, true),
                             vec("loss", loss, 1, 4, true),
                             vec("rewards", rewards, 2 * pairs, 4, true, true),
                             vec("dlogp", dlogp, tokens, 4, true, true)};
    if (need) ops.push_back(vec("workspace", workspace, int64_t(need / 8), 8, true));
    MUON_TRY(muon::check_operands(ops, d));
    muon::PrefArgs a{};
    a.logp = logp; a.ref = ref_logp; a.valid = valid; a.offsets = offsets; a.weight = weight; a.dloss = dloss;
    a.tokens = tokens; a.pairs = pairs;
    a.beta = beta; a.margin = margin; a.smoothing = smoothing; a.average = average;
    a.loss = loss; a.rewards = rewards; a.dlogp = dlogp;
    a.lone = muon::pref_lone(tokens, pairs);
    a.shift = muon::pref_shift(tokens, pairs);
    a.part = (double*)workspace;
    return launched(muon::run_preference_loss(a, (hipStream_t)stream));
  });
}

}  // extern "C"
