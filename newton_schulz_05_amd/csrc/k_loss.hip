// Clipped policy loss with a KL term, and the preference loss on pairs of
// answers, each with its gradient by the tokens' log-probabilities.
//
// A token's terms are differences of numbers near one another (e^u - u - 1 next
// to u = 0, d against the clipping border) and there is one of them for a whole
// row of logits, so everything here is fp64: the sums are exact to far below an
// fp32 step whatever their order, which is fixed all the same.
#include "ops_dev.hpp"

namespace muon {

namespace {

template <int WG> __device__ __forceinline__ double block_sum(double v, double* red) {
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x / 64] = v;
  __syncthreads();
  double s = red[0];
#pragma unroll
  for (int w = 1; w < WG / 64; ++w) s += red[w];
  return s;
}

// ---- policy loss ---------------------------------------------------------------

__device__ __forceinline__ void put_policy(const PolicyArgs& a, double pg, double kl, double cut) {
  a.loss[0] = float(pg + a.beta * kl);
  if (a.terms) {
    a.terms[0] = float(pg);
    a.terms[1] = float(kl);
    a.terms[2] = float(cut);
  }
}

constexpr int kPolicyThreads = 1024;
__global__ __launch_bounds__(kPolicyThreads) void policy_kernel(PolicyArgs a) {
  __shared__ double red[kPolicyThreads / 64];
  const double up = a.dloss ? double(a.dloss[0]) : 1.0;
  double sum_pg = 0.0, sum_kl = 0.0, sum_cut = 0.0;
  for (int64_t i = int64_t(blockIdx.x) * kPolicyThreads + threadIdx.x; i < a.tokens;
       i += int64_t(gridDim.x) * kPolicyThreads) {
    const double w = a.weight ? double(a.weight[i]) : 1.0, lp = a.logp[i], adv = a.adv[i];
    const double d = a.old_logp ? lp - double(a.old_logp[i]) : 0.0;
    const double u = a.ref ? double(a.ref[i]) - lp : 0.0;
    const bool cut = (adv > 0.0 && d > a.log_high) || (adv < 0.0 && d < a.log_low);
    const double gain = adv == 0.0 ? 0.0 : adv * exp(d), e = a.ref ? expm1(u) : 0.0;
    const double pg = cut ? -adv * (adv > 0.0 ? a.high : a.low) : -gain;
    if (w != 0.0) {
      sum_pg += w * pg;
      sum_kl += w * (e - u);
      sum_cut += cut ? w : 0.0;
    }
    if (a.dlogp) a.dlogp[i] = w != 0.0 ? float(up * w * ((cut ? 0.0 : -gain) - a.beta * e)) : 0.0f;
  }
  sum_pg = block_sum<kPolicyThreads>(sum_pg, red);
  sum_kl = block_sum<kPolicyThreads>(sum_kl, red);
  sum_cut = block_sum<kPolicyThreads>(sum_cut, red);
  if (threadIdx.x != 0) return;
  if (a.parts == 1) {
    put_policy(a, sum_pg, sum_kl, sum_cut);
  } else {
    double* to = a.part + int64_t(blockIdx.x) * 3;
    to[0] = sum_pg;
    to[1] = sum_kl;
    to[2] = sum_cut;
  }
}

__global__ __launch_bounds__(kPolicyMaxParts) void policy_join_kernel(PolicyArgs a) {
  __shared__ double red[kPolicyMaxParts / 64];
  const bool have = int(threadIdx.x) < a.parts;
  const double* from = a.part + threadIdx.x * 3;
  const double pg = block_sum<kPolicyMaxParts>(have ? from[0] : 0.0, red);
  const double kl = block_sum<kPolicyMaxParts>(have ? from[1] : 0.0, red);
  const double cut = block_sum<kPolicyMaxParts>(have ? from[2] : 0.0, red);
  if (threadIdx.x == 0) put_policy(a, pg, kl, cut);
}

// ---- preference loss -------------------------------------------------------------

constexpr int kPrefThreads = 256;

// Tokens of chunk c of sequence s.
struct Run {
  int64_t from, to;
};
__device__ __forceinline__ Run run_of(const PrefArgs& a, int64_t s, int c) {
  auto in = [&](int64_t v) { return v < 0 ? 0 : v > a.tokens ? a.tokens : v; };
  const int64_t b = in(a.offsets[s]), e = in(a.offsets[s + 1]), n = e > b ? e - b : 0;
  const int64_t each = (n + a.chunks - 1) / a.chunks, from = each * c < n ? each * c : n;
  return {b + from, b + (from + each < n ? from + each : n)};
}

__global__ __launch_bounds__(kPrefThreads) void pref_sum_kernel(PrefArgs a) {
  __shared__ double red[kPrefThreads / 64];
  const int64_t s = blockIdx.x;
  const Run r = run_of(a, s, int(blockIdx.y));
  double sum = 0.0, count = 0.0;
  for (int64_t i = r.from + threadIdx.x; i < r.to; i += kPrefThreads) {
    const bool in = !a.valid || a.valid[i] != 0;
    if (in) {
      sum += a.ref ? double(a.logp[i]) - double(a.ref[i]) : double(a.logp[i]);
      count += 1.0;
    }
  }
  sum = block_sum<kPrefThreads>(sum, red);
  count = block_sum<kPrefThreads>(count, red);
  if (threadIdx.x == 0) {
    double* to = a.part + (s * a.chunks + blockIdx.y) * 2;
    to[0] = sum;
    to[1] = count;
  }
}

// Reward of a sequence and what multiplies a token's gradient.
struct Reward {
  double r, share;
};
__device__ __forceinline__ Reward reward(const PrefArgs& a, int64_t s) {
  double sum = 0.0, count = 0.0;
  for (int c = 0; c < a.chunks; ++c) {
    sum += a.part[(s * a.chunks + c) * 2];
    count += a.part[(s * a.chunks + c) * 2 + 1];
  }
  const double share = a.average ? (count > 0.0 ? a.beta / count : 0.0) : a.beta;
  return {share * sum, share};
}

// log(1 + e^x)
__device__ __forceinline__ double softplus(double x) { return (x > 0.0 ? x : 0.0) + log1p(exp(-fabs(x))); }

__global__ __launch_bounds__(kPrefThreads) void pref_grad_kernel(PrefArgs a) {
  __shared__ double red[kPrefThreads / 64];
  if (int64_t(blockIdx.x) == 2 * a.pairs) {  // the loss
    if (blockIdx.y != 0) return;
    double loss = 0.0;
    for (int64_t i = threadIdx.x; i < a.pairs; i += kPrefThreads) {
      const Reward x = reward(a, i), y = reward(a, a.pairs + i);
      const double m = x.r - y.r - a.margin, w = a.weight ? double(a.weight[i]) : 1.0 / double(a.pairs);
      if (w != 0.0) loss += w * ((1.0 - a.smoothing) * softplus(-m) + a.smoothing * softplus(m));
      if (a.rewards) {
        a.rewards[i] = float(x.r);
        a.rewards[a.pairs + i] = float(y.r);
      }
    }
    loss = block_sum<kPrefThreads>(loss, red);
    if (threadIdx.x == 0) a.loss[0] = float(loss);
    return;
  }
  const int64_t s = blockIdx.x, pair = s < a.pairs ? s : s - a.pairs;
  const Run r = run_of(a, s, int(blockIdx.y));
  if (!a.dlogp || r.from >= r.to) return;
  const Reward x = reward(a, pair), y = reward(a, a.pairs + pair);
  const double m = x.r - y.r - a.margin, w = a.weight ? double(a.weight[pair]) : 1.0 / double(a.pairs);
  const double up = a.dloss ? double(a.dloss[0]) : 1.0;
  // d loss / d m = w (smoothing sigma(m) - (1 - smoothing) sigma(-m))
  const double slope = w * (a.smoothing / (1.0 + exp(-m)) - (1.0 - a.smoothing) / (1.0 + exp(m)));
  const float g = w != 0.0 ? float(up * slope * (s < a.pairs ? x.share : -y.share)) : 0.0f;
  for (int64_t i = r.from + threadIdx.x; i < r.to; i += kPrefThreads)
    a.dlogp[i] = !a.valid || a.valid[i] != 0 ? g : 0.0f;
}

}  // namespace

hipError_t run_policy_loss(const PolicyArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(policy_kernel, dim3(unsigned(a.parts)), dim3(kPolicyThreads), 0, st, a);
  if (a.parts > 1) hipLaunchKernelGGL(policy_join_kernel, dim3(1), dim3(kPolicyMaxParts), 0, st, a);
  return hipGetLastError();
}

hipError_t run_preference_loss(const PrefArgs& a, hipStream_t st) {
  const unsigned seqs = unsigned(2 * a.pairs);
  if (seqs > 0)
    hipLaunchKernelGGL(pref_sum_kernel, dim3(seqs, unsigned(a.chunks)), dim3(kPrefThreads), 0, st, a);
  // without a gradient only the workgroup of the loss is left
  hipLaunchKernelGGL(pref_grad_kernel, dim3(seqs + 1, unsigned(a.dlogp ? a.chunks : 1)), dim3(kPrefThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace muon
