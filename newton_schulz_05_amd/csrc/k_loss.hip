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

// Sums of N values over a workgroup, in a fixed order; in every thread.
template <int WG, int N> __device__ __forceinline__ void block_sum(double (&v)[N], double (*red)[N]) {
  for (int d = 32; d >= 1; d >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], d, 64);
  }
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[threadIdx.x / 64][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = red[0][i];
#pragma unroll
    for (int w = 1; w < WG / 64; ++w) v[i] += red[w][i];
  }
}

// ---- policy loss ---------------------------------------------------------------

// Policy sum, KL sum and the weight of the clipped tokens.
__device__ __forceinline__ void put_policy(const PolicyArgs& a, const double (&s)[3]) {
  a.loss[0] = float(s[0] + a.beta * s[1]);
  if (a.terms) {
#pragma unroll
    for (int i = 0; i < 3; ++i) a.terms[i] = float(s[i]);
  }
}

constexpr int kPolicyThreads = 1024;
__global__ __launch_bounds__(kPolicyThreads) void policy_kernel(PolicyArgs a) {
  __shared__ double red[kPolicyThreads / 64][3];
  const double up = a.dloss ? double(a.dloss[0]) : 1.0;
  double sum[3] = {0.0, 0.0, 0.0};
  for (int64_t i = int64_t(blockIdx.x) * kPolicyThreads + threadIdx.x; i < a.tokens;
       i += int64_t(gridDim.x) * kPolicyThreads) {
    const double w = a.weight ? double(a.weight[i]) : 1.0, lp = a.logp[i], adv = a.adv[i];
    const double d = a.old_logp ? lp - double(a.old_logp[i]) : 0.0;
    const double u = a.ref ? double(a.ref[i]) - lp : 0.0;
    const bool cut = (adv > 0.0 && d > a.log_high) || (adv < 0.0 && d < a.log_low);
    const double gain = adv == 0.0 ? 0.0 : adv * exp(d), e = a.ref ? expm1(u) : 0.0;
    const double pg = cut ? -adv * (adv > 0.0 ? a.high : a.low) : -gain;
    if (w != 0.0) {
      sum[0] += w * pg;
      sum[1] += w * (e - u);
      sum[2] += cut ? w : 0.0;
    }
    if (a.dlogp) a.dlogp[i] = w != 0.0 ? float(up * w * ((cut ? 0.0 : -gain) - a.beta * e)) : 0.0f;
  }
  block_sum<kPolicyThreads>(sum, red);
  if (threadIdx.x != 0) return;
  if (a.parts == 1) {
    put_policy(a, sum);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i) a.part[int64_t(blockIdx.x) * 3 + i] = sum[i];
  }
}

__global__ __launch_bounds__(kPolicyMaxParts) void policy_join_kernel(PolicyArgs a) {
  __shared__ double red[kPolicyMaxParts / 64][3];
  double sum[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) sum[i] = int(threadIdx.x) < a.parts ? a.part[threadIdx.x * 3 + i] : 0.0;
  block_sum<kPolicyMaxParts>(sum, red);
  if (threadIdx.x == 0) put_policy(a, sum);
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

// Four tokens at i (those before n), 0 behind.
__device__ __forceinline__ f32x4 load4(const float* p, int64_t i, int64_t n) {
  if (i + 4 <= n) return *(const f32x4_u*)(p + i);
  f32x4 v{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n) v[j] = p[i + j];
  return v;
}
__device__ __forceinline__ bool counts(const PrefArgs& a, int64_t i) { return !a.valid || a.valid[i] != 0; }

__global__ __launch_bounds__(kPrefThreads) void pref_sum_kernel(PrefArgs a) {
  __shared__ double red[kPrefThreads / 64][2];
  const int64_t s = blockIdx.x;
  const Run r = run_of(a, s, int(blockIdx.y));
  double sum[2] = {0.0, 0.0};  // and the number of tokens
  for (int64_t i = r.from + threadIdx.x * 4; i < r.to; i += kPrefThreads * 4) {
    const f32x4 x = load4(a.logp, i, r.to), y = a.ref ? load4(a.ref, i, r.to) : f32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < r.to && counts(a, i + j)) {
        sum[0] += double(x[j]) - double(y[j]);
        sum[1] += 1.0;
      }
  }
  block_sum<kPrefThreads>(sum, red);
  if (threadIdx.x == 0) {
    double* to = a.part + (s * a.chunks + blockIdx.y) * 2;
    to[0] = sum[0];
    to[1] = sum[1];
  }
}

// Reward of a sequence and what multiplies a token's gradient, from the sum and
// the number of its tokens.
struct Reward {
  double r, share;
};
__device__ __forceinline__ Reward reward(const PrefArgs& a, double sum, double count) {
  const double share = a.average ? (count > 0.0 ? a.beta / count : 0.0) : a.beta;
  return {share * sum, share};
}
// A pair's rewards: by one thread, or by a wave with a chunk a lane (in every
// lane; 64 chunks one after the other took 5 us of a workgroup).
struct Pair {
  Reward x, y;
  double m, w;
};
template <bool WAVE> __device__ __forceinline__ Pair pair_of(const PrefArgs& a, int64_t i) {
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  const double *p = a.part + i * a.chunks * 2, *q = a.part + (a.pairs + i) * a.chunks * 2;
  auto add = [&](int c) {
    s[0] += p[2 * c];
    s[1] += p[2 * c + 1];
    s[2] += q[2 * c];
    s[3] += q[2 * c + 1];
  };
  if constexpr (WAVE) {
    static_assert(kPrefMaxChunks == 64);
    const int lane = threadIdx.x & 63;
    if (lane < a.chunks) add(lane);
    for (int d = 32; d >= 1; d >>= 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += __shfl_xor(s[k], d, 64);
    }
  } else {
    for (int c = 0; c < a.chunks; ++c) add(c);
  }
  Pair r;
  r.x = reward(a, s[0], s[1]);
  r.y = reward(a, s[2], s[3]);
  r.m = r.x.r - r.y.r - a.margin;
  r.w = a.weight ? double(a.weight[i]) : 1.0 / double(a.pairs);
  return r;
}

// log(1 + e^x)
__device__ __forceinline__ double softplus(double x) { return (x > 0.0 ? x : 0.0) + log1p(exp(-fabs(x))); }

// The loss, by one workgroup; a pair's rewards come with it.
template <bool WAVE> __device__ __forceinline__ void pref_loss(const PrefArgs& a, double (*red)[1]) {
  constexpr int EACH = WAVE ? 64 : 1;
  const bool first = threadIdx.x % EACH == 0;
  double loss[1] = {0.0};
  for (int64_t i = threadIdx.x / EACH; i < a.pairs; i += kPrefThreads / EACH) {
    const Pair p = pair_of<WAVE>(a, i);
    if (!first) continue;
    if (p.w != 0.0) loss[0] += p.w * ((1.0 - a.smoothing) * softplus(-p.m) + a.smoothing * softplus(p.m));
    if (a.rewards) {
      a.rewards[i] = float(p.x.r);
      a.rewards[a.pairs + i] = float(p.y.r);
    }
  }
  block_sum<kPrefThreads>(loss, red);
  if (threadIdx.x == 0) a.loss[0] = float(loss[0]);
}

// A few chunks are added by one thread for each pair.
constexpr int kFewChunks = 8;

__global__ __launch_bounds__(kPrefThreads) void pref_grad_kernel(PrefArgs a) {
  __shared__ double red[kPrefThreads / 64][1];
  if (int64_t(blockIdx.x) == 2 * a.pairs) {
    if (blockIdx.y != 0) return;
    if (a.chunks <= kFewChunks) pref_loss<false>(a, red);
    else pref_loss<true>(a, red);
    return;
  }
  const int64_t s = blockIdx.x, pair = s < a.pairs ? s : s - a.pairs;
  const Run r = run_of(a, s, int(blockIdx.y));
  if (!a.dlogp || r.from >= r.to) return;
  const Pair p = a.chunks <= kFewChunks ? pair_of<false>(a, pair) : pair_of<true>(a, pair);
  const double up = a.dloss ? double(a.dloss[0]) : 1.0;
  // d loss / d m = w (smoothing sigma(m) - (1 - smoothing) sigma(-m))
  const double slope = p.w * (a.smoothing / (1.0 + exp(-p.m)) - (1.0 - a.smoothing) / (1.0 + exp(p.m)));
  const float g = p.w != 0.0 ? float(up * slope * (s < a.pairs ? p.x.share : -p.y.share)) : 0.0f;
  for (int64_t i = r.from + threadIdx.x * 4; i < r.to; i += kPrefThreads * 4) {
    if (i + 4 <= r.to && !a.valid) {
      *(f32x4_u*)(a.dlogp + i) = f32x4{g, g, g, g};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < r.to) a.dlogp[i + j] = counts(a, i + j) ? g : 0.0f;
    }
  }
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
