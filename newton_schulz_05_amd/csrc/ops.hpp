// Host-side launch interface of the training operators beside the step:
// layer norm, dropout, the two fused, the expert router, the norm and rotation of
// query and key heads, token log-probabilities and the losses on them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_limits.hpp"

namespace muon {

// Counter-based dropout (Philox4x32-10, see ops_dev.hpp): an element is kept
// when its 16-bit draw is >= thresh, and then multiplied by scale.
struct DropArgs {
  uint32_t thresh;             // round(65536 p), 0 .. 65536
  float scale;                 // 65536 / (65536 - thresh), 0 when nothing is kept
  uint32_t k0, k1;             // seed
  uint64_t offset;             // stream position, added to *offset_dev
  const uint64_t* offset_dev;  // device word, or null
};

struct NormFwdArgs {
  const void* x;      // [rows, cols]
  const void* res;    // fused: residual
  void* h;            // fused: residual + dropout(x)
  void* y;
  const void* gamma;  // null: 1
  const void* beta;   // null: 0
  float* mean;        // null: not stored
  float* rstd;
  int64_t rows, ld_x, ld_res, ld_h, ld_y;
  int cols;
  float eps;
  DropArgs drop;
};

struct NormBwdArgs {
  const void* dy;
  const void* x;      // the norm's input (fused: h)
  const void* dh;     // fused: gradient that reaches h by the residual path, or null
  const void* gamma;  // null: 1
  const float* mean;
  const float* rstd;
  void* dx;           // fused: gradient of the dropped-out input
  void* dres;         // fused: gradient of h, which is the residual's
  void* dgamma;       // null: not wanted
  void* dbeta;
  float* part;        // [parts][2][cols] partial sums of dgamma and dbeta
  int parts;
  int64_t rows, ld_dy, ld_x, ld_dh, ld_dx, ld_dres;
  int cols;
  DropArgs drop;
};

struct DropoutArgs {
  const void* x;
  const void* res;  // or null
  void* out;
  int64_t rows, cols, ld_x, ld_res, ld_out;
  DropArgs drop;
};

struct RouteArgs {
  const void* logits;
  const uint8_t* valid;  // or null: every token counts
  int64_t rows, ld;
  int experts, k;
  int renorm;
  float coef;
  int32_t* idx;
  float* gates;
  int32_t* counts;
  int32_t* n_tokens;
  float* prob_mean;  // or null
  float* loss;
  float* part_p;     // [parts][experts]
  int32_t* part_c;   // [parts][experts]
  int32_t* part_n;   // [parts]
  int parts;
  double* terms;     // the loss's, one for each 16 experts
  uint32_t* ticket;  // workgroups that have added theirs
};

struct RouteBwdArgs {
  const void* logits;
  const uint8_t* valid;
  int64_t rows, ld, ld_d;
  int experts, k;
  int renorm;
  float coef;
  const int32_t* idx;
  const int32_t* counts;
  const int32_t* n_tokens;
  const float* dgates;  // or null: 0
  const float* dloss;   // or null: 1
  void* dlogits;
};

// The heads of queries or of keys as rows, in the order of their input's
// memory: row r stands at (i0, i1, i2), i0 = r % n0, i1 = r / n0 % n1.
struct HeadRows {
  const void* x;
  const void* dy;     // backward
  void* out;          // forward: y; backward: dx
  const void* gamma;  // null: 1
  void* dgamma;       // null: not wanted
  float* part;        // [wgs][dim] partial sums of dgamma, or null
  FastDiv n0, n1;
  int64_t s_x[3], s_dy[3], s_out[3];
  int64_t s_pos[3];   // of the word of positions, or of the table's row
  uint32_t rows;
  int wgs;            // workgroups that take these rows
};

struct HeadArgs {
  HeadRows q, k;
  const float* cos;
  const float* sin;
  const int64_t* positions;  // null: s_pos leads to the table's row itself
  int64_t table_rows;
  int dim, rot;
  float eps;
  bool wbf16;
  bool stream_out;           // outputs that the caches do not hold
};

struct LogpArgs {
  const void* logits;
  const int64_t* targets;
  int64_t rows, cols, ld;
  float scale, scale2;  // scale2 = scale log2(e)
  float* logp;
  float* lse;
  int parts;
  float* part;          // [rows][parts][2]: maximum and sum
};

struct LogpBwdArgs {
  const void* logits;
  const int64_t* targets;
  int64_t rows, cols, ld, ld_d;
  float scale, scale2;
  const float* logp;
  const float* lse;
  const float* dlogp;
  void* dlogits;
  bool stream_out, in_place;
};

struct PolicyArgs {
  const float* logp;
  const float* old_logp;  // null: logp
  const float* ref;       // null: no KL term
  const float* adv;
  const float* weight;    // null: 1
  const float* dloss;     // null: 1
  int64_t tokens;
  double low, high;           // 1 - clip_low, 1 + clip_high
  double log_low, log_high;
  double beta;
  float* loss;
  float* terms;           // or null
  float* dlogp;           // or null
  int parts;
  double* part;           // [parts][3]
};

struct PrefArgs {
  const float* logp;
  const float* ref;      // null: 0
  const uint8_t* valid;  // null: every token counts
  const int64_t* offsets;
  const float* weight;   // null: 1 / pairs
  const float* dloss;    // null: 1
  int64_t tokens, pairs;
  double beta, margin, smoothing;
  int average;
  float* loss;
  float* rewards;        // or null
  float* dlogp;          // or null
  bool lone;             // one workgroup takes all
  int shift;             // else 2^shift workgroups take a sequence
  double* part;          // [2 pairs][2^shift][2]: sum and number of tokens
};

// `bf16`: element type of the activations, `wbf16`: of gamma and beta.
hipError_t run_norm_fwd(const NormFwdArgs& a, bool bf16, bool wbf16, bool fused, hipStream_t st);
hipError_t run_norm_bwd(const NormBwdArgs& a, bool bf16, bool wbf16, bool fused, hipStream_t st);
hipError_t run_dropout(const DropoutArgs& a, bool bf16, hipStream_t st);
hipError_t run_route_fwd(const RouteArgs& a, bool bf16, hipStream_t st);
hipError_t run_route_bwd(const RouteBwdArgs& a, bool bf16, hipStream_t st);
hipError_t run_heads_fwd(const HeadArgs& a, bool bf16, bool interleaved, hipStream_t st);
hipError_t run_heads_bwd(const HeadArgs& a, bool bf16, bool interleaved, hipStream_t st);
hipError_t run_logp_fwd(const LogpArgs& a, bool bf16, hipStream_t st);
hipError_t run_logp_bwd(const LogpBwdArgs& a, bool bf16, hipStream_t st);
hipError_t run_policy_loss(const PolicyArgs& a, hipStream_t st);
hipError_t run_preference_loss(const PrefArgs& a, hipStream_t st);

}  // namespace muon
