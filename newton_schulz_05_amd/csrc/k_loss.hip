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

// A term that a factor of 0 takes out, an infinite one too.
__device__ __forceinline__ double scaled(double f, double v) { return f != 0.0 ? f * v : 0.0; }

// ---- policy loss ---------------------------------------------------------------

// Policy sum, KL sum and the weight of the clipped tokens.
__device__ __forceinline__ void put_policy(const PolicyArgs& a, const double (&s)[3]) {
  a.loss[0] = float(s[0] + scaled(a.beta, s[1]));
  if (a.terms) {
#pragma unroll
    for (int i = 0; i < 3; ++i) a.terms[i] = float(s[i]);
  }
}

// A token a thread at a time; the workgroups' sums are joined by a second launch.
// Launches and latency: 777 tokens 3.8 us, 262144 5.6 and 1.6 for the join (1.2 us
// of bytes), a million 12.2.  With a reduction for each of the three sums instead
// of one for all the 262144 took 6.9 and 2.2.
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
      sum[1] += w * (u == INFINITY ? u : e - u);
      sum[2] += cut ? w : 0.0;
    }
    if (a.dlogp) a.dlogp[i] = w != 0.0 ? float(up * w * ((cut ? 0.0 : -gain) - scaled(a.beta, e))) : 0.0f;
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

struct Run {
  int64_t from, to;
};
// Tokens of sequence s, and of chunk c of it.
__device__ __forceinline__ Run run_of(const PrefArgs& a, int64_t s) {
  auto in = [&](int64_t v) { return v < 0 ? 0 : v > a.tokens ? a.tokens : v; };
  const int64_t b = in(a.offsets[s]), e = in(a.offsets[s + 1]);
  return {b, e > b ? e : b};
}
__device__ __forceinline__ Run run_of(const PrefArgs& a, int64_t s, int c) {
  const Run r = run_of(a, s);
  const int64_t n = r.to - r.from, each = (n + (1 << a.shift) - 1) >> a.shift, from = each * c < n ? each * c : n;
  return {r.from + from, r.from + (from + each < n ? from + each : n)};
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

// What thread t of `threads` adds of a run: the sum, and the number of tokens.
__device__ __forceinline__ void add_run(const PrefArgs& a, const Run& r, int t, int threads, double (&sum)[2]) {
  sum[0] = sum[1] = 0.0;
#pragma unroll 2
  for (int64_t i = r.from + t * 4; i < r.to; i += threads * 4) {
    const f32x4 x = load4(a.logp, i, r.to), y = a.ref ? load4(a.ref, i, r.to) : f32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < r.to && counts(a, i + j)) {
        sum[0] += double(x[j]) - double(y[j]);
        sum[1] += 1.0;
      }
  }
}
__device__ __forceinline__ void put_run(const PrefArgs& a, const Run& r, int t, int threads, float g) {
  for (int64_t i = r.from + t * 4; i < r.to; i += threads * 4) {
    if (i + 4 <= r.to && !a.valid) {
      *(f32x4_u*)(a.dlogp + i) = f32x4{g, g, g, g};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < r.to) a.dlogp[i + j] = counts(a, i + j) ? g : 0.0f;
    }
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
struct Pair {
  Reward x, y;
  double m, w;
};
__device__ __forceinline__ Pair pair_of(const PrefArgs& a, int64_t i, const double* x, const double* y) {
  Pair p;
  p.x = reward(a, x[0], x[1]);
  p.y = reward(a, y[0], y[1]);
  p.m = p.x.r - p.y.r - a.margin;
  p.w = a.weight ? double(a.weight[i]) : 1.0 / double(a.pairs);
  return p;
}
// Gradient of a token of the pair's first or second sequence:
// d loss / d m = w (smoothing sigma(m) - (1 - smoothing) sigma(-m)).
__device__ __forceinline__ float gradient(const PrefArgs& a, const Pair& p, bool first) {
  const double up = a.dloss ? double(a.dloss[0]) : 1.0;
  const double slope = p.w * (a.smoothing / (1.0 + exp(-p.m)) - (1.0 - a.smoothing) / (1.0 + exp(p.m)));
  return p.w != 0.0 ? float(up * slope * (first ? p.x.share : -p.y.share)) : 0.0f;
}
// log(1 + e^x)
__device__ __forceinline__ double softplus(double x) { return (x > 0.0 ? x : 0.0) + log1p(exp(-fabs(x))); }
// The pair's part of the loss; its rewards come with it.
__device__ __forceinline__ double put_pair(const PrefArgs& a, int64_t i, const Pair& p) {
  if (a.rewards) {
    a.rewards[i] = float(p.x.r);
    a.rewards[a.pairs + i] = float(p.y.r);
  }
  return p.w != 0.0 ? p.w * (scaled(1.0 - a.smoothing, softplus(-p.m)) + scaled(a.smoothing, softplus(p.m))) : 0.0;
}

// 96 pairs of 4096 tokens: 5.4 us, and 5.7 for pref_grad_kernel, where the bytes
// take 1.8; both are launch and latency.  With 2048 tokens a chunk instead of 512
// the longest answers' workgroups took 14.6.
__global__ __launch_bounds__(kPrefThreads) void pref_sum_kernel(PrefArgs a) {
  __shared__ double red[kPrefThreads / 64][2];
  const int64_t s = blockIdx.x;
  double sum[2];
  add_run(a, run_of(a, s, int(blockIdx.y)), threadIdx.x, kPrefThreads, sum);
  block_sum<kPrefThreads>(sum, red);
  if (threadIdx.x == 0) {
    double* to = a.part + ((s << a.shift) + blockIdx.y) * 2;
    to[0] = sum[0];
    to[1] = sum[1];
  }
}

// A pair from its chunks' sums: by one thread, or by a wave with a chunk a lane
// (in every lane; 64 chunks one after the other took 5 us of a workgroup).
template <bool WAVE> __device__ __forceinline__ Pair pair_of(const PrefArgs& a, int64_t i) {
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  const double *p = a.part + (i << a.shift) * 2, *q = a.part + ((a.pairs + i) << a.shift) * 2;
  auto add = [&](int c) {
    s[0] += p[2 * c];
    s[1] += p[2 * c + 1];
    s[2] += q[2 * c];
    s[3] += q[2 * c + 1];
  };
  if constexpr (WAVE) {
    static_assert(kPrefMaxChunks == 64);
    const int lane = threadIdx.x & 63;
    if (lane < (1 << a.shift)) add(lane);
    for (int d = 32; d >= 1; d >>= 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += __shfl_xor(s[k], d, 64);
    }
  } else {
    for (int c = 0; c < (1 << a.shift); ++c) add(c);
  }
  return pair_of(a, i, s, s + 2);
}

// The loss, by one workgroup.
template <bool WAVE> __device__ __forceinline__ void pref_loss(const PrefArgs& a, double (*red)[1]) {
  constexpr int EACH = WAVE ? 64 : 1;
  double loss[1] = {0.0};
  for (int64_t i = threadIdx.x / EACH; i < a.pairs; i += kPrefThreads / EACH) {
    const Pair p = pair_of<WAVE>(a, i);
    if (threadIdx.x % EACH == 0) loss[0] += put_pair(a, i, p);
  }
  block_sum<kPrefThreads>(loss, red);
  if (threadIdx.x == 0) a.loss[0] = float(loss[0]);
}

// Up to 8 chunks are added by one thread for each pair.
constexpr int kFewShift = 3;

__global__ __launch_bounds__(kPrefThreads) void pref_grad_kernel(PrefArgs a) {
  __shared__ double red[kPrefThreads / 64][1];
  __shared__ float grad;
  if (int64_t(blockIdx.x) == 2 * a.pairs) {
    if (blockIdx.y != 0) return;
    if (a.shift <= kFewShift) pref_loss<false>(a, red);
    else pref_loss<true>(a, red);
    return;
  }
  if (!a.dlogp) return;
  const int64_t s = blockIdx.x;
  const Run r = run_of(a, s, int(blockIdx.y));
  if (threadIdx.x < 64) {  // by one wave: the fp64 exponentials of four took half of the kernel
    const Pair p = pair_of<true>(a, s < a.pairs ? s : s - a.pairs);
    if (threadIdx.x == 0) grad = gradient(a, p, s < a.pairs);
  }
  __syncthreads();
  put_run(a, r, threadIdx.x, kPrefThreads, grad);
}

// Few pairs of few tokens: one workgroup, a wave a sequence (4 pairs of 300 5.2 us
// in a graph, 5.8 with two launches, and 4 us less on the host).
__global__ __launch_bounds__(1024) void pref_lone_kernel(PrefArgs a) {
  static_assert(2 * kPrefLonePairs <= 16);
  __shared__ double sums[16][2];
  __shared__ double terms[kPrefLonePairs];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int pairs = int(a.pairs);
  Run r{0, 0};
  if (wave < 2 * pairs) {
    r = run_of(a, wave);
    double sum[2];
    add_run(a, r, lane, 64, sum);
    for (int d = 32; d >= 1; d >>= 1) {
      sum[0] += __shfl_xor(sum[0], d, 64);
      sum[1] += __shfl_xor(sum[1], d, 64);
    }
    if (lane < 2) sums[wave][lane] = sum[lane];
  }
  __syncthreads();
  if (wave < 2 * pairs) {
    const int i = wave < pairs ? wave : wave - pairs;
    const Pair p = pair_of(a, i, sums[i], sums[pairs + i]);
    if (wave < pairs && lane == 0) terms[i] = put_pair(a, i, p);
    if (a.dlogp) put_run(a, r, lane, 64, gradient(a, p, wave < pairs));
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double loss = 0.0;
    for (int i = 0; i < pairs; ++i) loss += terms[i];
    a.loss[0] = float(loss);
  }
}

}  // namespace

hipError_t run_policy_loss(const PolicyArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(policy_kernel, dim3(unsigned(a.parts)), dim3(kPolicyThreads), 0, st, a);
  if (a.parts > 1) hipLaunchKernelGGL(policy_join_kernel, dim3(1), dim3(kPolicyMaxParts), 0, st, a);
  return hipGetLastError();
}

hipError_t run_preference_loss(const PrefArgs& a, hipStream_t st) {
  if (a.lone) {
    hipLaunchKernelGGL(pref_lone_kernel, dim3(1), dim3(1024), 0, st, a);
    return hipGetLastError();
  }
  const unsigned seqs = unsigned(2 * a.pairs), chunks = 1u << a.shift;
  if (seqs > 0) hipLaunchKernelGGL(pref_sum_kernel, dim3(seqs, chunks), dim3(kPrefThreads), 0, st, a);
  // without a gradient only the workgroup of the loss is left
  hipLaunchKernelGGL(pref_grad_kernel, dim3(seqs + 1, a.dlogp ? chunks : 1), dim3(kPrefThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace muon
