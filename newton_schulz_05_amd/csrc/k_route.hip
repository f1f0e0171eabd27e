// Expert router: softmax over the experts, the k largest as choices with
// their gates, the number of choices of every expert, and the balance loss
//   L = coef E sum_e f_e P_e,  f_e = c_e / (k n),  P_e = (1 / n) sum_t p_te
// over the n tokens that have a choice, with gradients through P and the
// gates (the counts c are constants):
//   dp_te = coef E c_e / (k n^2) dL + [e chosen] (gradient of its gate),
//   dlogit = p (dp - sum_e p dp).
// A group of 8 or 16 lanes holds one token's logits in registers, each lane
// PER consecutive experts, so the maximum, the sums and the choices are
// reductions over at most 16 lanes, all of them single DPP steps.
#include "ops_dev.hpp"

#include <type_traits>

namespace muon {

namespace {

constexpr int WG = kRouteThreads;

// Order-preserving bits of a float: larger value, larger word; 0 for -inf
// (an expert that is shut off), which is never chosen.  -0 counts as 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return v == -INFINITY ? 0u : u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

template <int N> __device__ __forceinline__ uint32_t lane_max(uint32_t v) {
  return lane_reduce<N>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int N> __device__ __forceinline__ uint32_t lane_min(uint32_t v) {
  return lane_reduce<N>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

// The PER logits of experts base .. base + PER - 1 (-inf behind the last one).
template <typename T, int PER>
__device__ __forceinline__ void load_logits(const T* p, int n, float (&v)[PER]) {
  if constexpr (PER >= 8) {
#pragma unroll
    for (int i = 0; i < PER; i += 8) {
      float w[8];
      unpack8(load8(p + i, n - i), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i + j] = i + j < n ? w[j] : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = i < n ? Elem<T>::load(p + i) : -INFINITY;
  }
}

template <typename T, int LANES, int PER>
__global__ __launch_bounds__(WG) void route_fwd_kernel(RouteArgs a) {
  constexpr int TOK = WG / LANES;
  __shared__ int32_t hist[LANES * PER];
  __shared__ float sums[WG / 64][LANES * PER];
  __shared__ int32_t ntok;
  const int t = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  const int base = t * PER, mine = a.experts - base;
  for (int e = threadIdx.x; e < LANES * PER; e += WG) hist[e] = 0;
  if (threadIdx.x == 0) ntok = 0;
  __syncthreads();
  float psum[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) psum[i] = 0.0f;
  int n = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * TOK; row0 < a.rows; row0 += int64_t(gridDim.x) * TOK) {
    const int64_t row = row0 + sub;
    const bool in = row < a.rows;
    const bool live = in && (!a.valid || a.valid[row] != 0);
    float v[PER];
    load_logits<T, PER>((const T*)a.logits + row * a.ld + base, live ? mine : 0, v);
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = order_key(v[i]);
    uint32_t top = 0, won = 0;
    int idx = -1;
    for (int j = 0; j < a.k; ++j) {
      uint32_t best = key[0], at = 0;
#pragma unroll
      for (int i = 1; i < PER; ++i) {
        at = key[i] > best ? i : at;
        best = key[i] > best ? key[i] : best;
      }
      const uint32_t m = lane_max<LANES>(best);
      if (j == 0) top = m;
      const uint32_t e = lane_min<LANES>(best == m ? base + at : 0xffffu);
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = base + i == int(e) ? 0u : key[i];
      if (t == j) {
        won = m;
        idx = m ? int(e) : -1;
      }
    }
    const bool some = top != 0;
    const float mx = some ? key_value(top) : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = expf(v[i] - mx);
      s += v[i];
    }
    const float total = lane_sum<LANES>(s);
    const float inv = some ? 1.0f / total : 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) psum[i] = fmaf(v[i], inv, psum[i]);
    float gate = idx >= 0 ? expf(key_value(won) - mx) * inv : 0.0f;
    if (a.renorm) {
      const float all = lane_sum<LANES>(gate);
      gate = some ? gate / all : 0.0f;
    }
    if (idx >= 0) atomicAdd(&hist[idx], 1);
    n += some && t == 0;
    if (in && t < a.k) {
      a.idx[row * a.k + t] = idx;
      a.gates[row * a.k + t] = gate;
    }
  }
  if (n) atomicAdd(&ntok, n);
  // the token groups of a wave, then the waves, in a fixed order
#pragma unroll
  for (int i = 0; i < PER; ++i) {
#pragma unroll
    for (int d = LANES; d < 64; d *= 2) psum[i] += __shfl_xor(psum[i], d, 64);
    if ((threadIdx.x & 63) < LANES) sums[threadIdx.x / 64][base + i] = psum[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += WG) {
    a.part_p[int64_t(blockIdx.x) * a.experts + e] = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
    a.part_c[int64_t(blockIdx.x) * a.experts + e] = hist[e];
  }
  if (threadIdx.x == 0) a.part_n[blockIdx.x] = ntok;
}

// Joins the workgroups' sums (one workgroup; thread (slice, e) takes every
// S-th partial sum of expert e, the slices are joined in order).
__global__ __launch_bounds__(1024) void route_join_kernel(RouteArgs a, int width) {
  __shared__ float sp[1024];
  __shared__ int32_t sc[1024];
  __shared__ double term[16];
  __shared__ int32_t ntok;
  const int e = threadIdx.x & (width - 1), slice = threadIdx.x / width, slices = 1024 / width;
  if (threadIdx.x == 0) ntok = 0;
  __syncthreads();
  int n = 0;
  for (int g = threadIdx.x; g < a.parts; g += 1024) n += a.part_n[g];
  if (n) atomicAdd(&ntok, n);
  float p = 0.0f;
  int32_t c = 0;
  if (e < a.experts)
    for (int g = slice; g < a.parts; g += slices) {
      p += a.part_p[int64_t(g) * a.experts + e];
      c += a.part_c[int64_t(g) * a.experts + e];
    }
  sp[threadIdx.x] = p;
  sc[threadIdx.x] = c;
  __syncthreads();
  const double tokens = ntok > 0 ? double(ntok) : 1.0;
  double x = 0.0;
  if (slice == 0 && e < a.experts) {
    for (int i = 1; i < slices; ++i) {
      p += sp[i * width + e];
      c += sc[i * width + e];
    }
    a.counts[e] = c;
    if (a.prob_mean) a.prob_mean[e] = float(double(p) / tokens);
    x = double(c) * double(p);
  }
  for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d, 64);
  if ((threadIdx.x & 63) == 0) term[threadIdx.x >> 6] = x;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 16; ++i) x += term[i];
    a.loss[0] = float(double(a.coef) * a.experts * x / (double(a.k) * tokens * tokens));
    a.n_tokens[0] = ntok;
  }
}

template <typename T, int LANES, int PER>
__global__ __launch_bounds__(WG) void route_bwd_kernel(RouteBwdArgs a) {
  constexpr int TOK = WG / LANES;
  const int t = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  const int base = t * PER, mine = a.experts - base;
  // A constant added to every dp of a token changes nothing (sum p = 1), so
  // the counts enter as E c_e - sum c, formed exactly in integers: near
  // balance the differences are what matters.
  int64_t c[PER], all = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] = i < mine ? a.counts[base + i] : 0;
    all += c[i];
  }
#pragma unroll
  for (int d = 1; d < LANES; d *= 2) all += __shfl_xor(all, d, 64);
  const int ntok = a.n_tokens[0];
  const double up = ntok > 0 ? double(a.coef) * (a.dloss ? double(a.dloss[0]) : 1.0) / (double(a.k) * ntok * ntok) : 0.0;
  float bal[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) bal[i] = float(up * double(c[i] * a.experts - all));
  for (int64_t row0 = int64_t(blockIdx.x) * TOK; row0 < a.rows; row0 += int64_t(gridDim.x) * TOK) {
    const int64_t row = row0 + sub;
    const bool in = row < a.rows;
    const bool live = in && (!a.valid || a.valid[row] != 0);
    float v[PER];
    load_logits<T, PER>((const T*)a.logits + row * a.ld + base, live ? mine : 0, v);
    float mx = v[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) mx = fmaxf(mx, v[i]);
    mx = lane_reduce<LANES>(mx, [](float x, float y) { return fmaxf(x, y); });
    const bool some = mx != -INFINITY;
    mx = some ? mx : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = expf(v[i] - mx);
      s += v[i];
    }
    const float total = lane_sum<LANES>(s);
    const float inv = some ? 1.0f / total : 0.0f;
    // lane t holds the token's choice t
    int idx = -1;
    float dg = 0.0f;
    if (live && a.dgates && t < a.k) {
      idx = a.idx[row * a.k + t];
      if (idx < 0 || idx >= a.experts) idx = -1;
      else dg = a.dgates[row * a.k + t];
    }
    if (a.dgates && a.renorm) {
      const float q = idx >= 0 ? expf(Elem<T>::load((const T*)a.logits + row * a.ld + idx) - mx) * inv : 0.0f;
      const float sum = lane_sum<LANES>(q);
      const float share = sum > 0.0f ? q / sum : 0.0f;  // exactly 1 for a lone choice, which has no gradient
      const float mid = lane_sum<LANES>(dg * share);
      dg = sum > 0.0f ? (dg - mid) / sum : 0.0f;
    }
    float dp[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) dp[i] = bal[i];
    if (a.dgates) {
      for (int j = 0; j < a.k; ++j) {
        const int e = __shfl(idx, j, LANES) - base;
        const float x = __shfl(dg, j, LANES);
#pragma unroll
        for (int i = 0; i < PER; ++i) dp[i] += e == i ? x : 0.0f;
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] *= inv;
      dot = fmaf(v[i], dp[i], dot);
    }
    dot = lane_sum<LANES>(dot);
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] *= dp[i] - dot;
    if (in) {
      T* out = (T*)a.dlogits + row * a.ld_d + base;
      if constexpr (PER >= 8) {
#pragma unroll
        for (int i = 0; i < PER; i += 8) {
          float w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = v[i + j];
          store8(out + i, mine - i, pack8(w, (const T*)nullptr));
        }
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i < mine) Elem<T>::store(out + i, v[i]);
      }
    }
  }
}

template <typename F> void by_experts(int experts, F f) {
  typedef std::integral_constant<int, 8> L8;
  typedef std::integral_constant<int, 16> L16;
  if (route_lanes(experts) == 8) f(L8{}, std::integral_constant<int, 1>{});
  else if (experts <= 16) f(L16{}, std::integral_constant<int, 1>{});
  else if (experts <= 32) f(L16{}, std::integral_constant<int, 2>{});
  else if (experts <= 64) f(L16{}, std::integral_constant<int, 4>{});
  else if (experts <= 128) f(L16{}, std::integral_constant<int, 8>{});
  else if (experts <= 256) f(L16{}, std::integral_constant<int, 16>{});
  else if (experts <= 512) f(L16{}, std::integral_constant<int, 32>{});
  else f(L16{}, std::integral_constant<int, 64>{});
}

}  // namespace

hipError_t run_route_fwd(const RouteArgs& a, bool bf16, hipStream_t st) {
  if (a.parts > 0)
    by_experts(a.experts, [&](auto lanes, auto per) {
      constexpr int L = decltype(lanes)::value, P = decltype(per)::value;
      if (bf16) hipLaunchKernelGGL((route_fwd_kernel<uint16_t, L, P>), dim3(unsigned(a.parts)), dim3(WG), 0, st, a);
      else hipLaunchKernelGGL((route_fwd_kernel<float, L, P>), dim3(unsigned(a.parts)), dim3(WG), 0, st, a);
    });
  int width = 1;
  while (width < a.experts) width *= 2;
  hipLaunchKernelGGL(route_join_kernel, dim3(1), dim3(1024), 0, st, a, width);
  return hipGetLastError();
}

hipError_t run_route_bwd(const RouteBwdArgs& a, bool bf16, hipStream_t st) {
  by_experts(a.experts, [&](auto lanes, auto per) {
    constexpr int L = decltype(lanes)::value, P = decltype(per)::value;
    const int64_t need = (a.rows + WG / L - 1) / (WG / L);
    const dim3 grid(unsigned(std::min<int64_t>(need, 2048)));
    if (bf16) hipLaunchKernelGGL((route_bwd_kernel<uint16_t, L, P>), grid, dim3(WG), 0, st, a);
    else hipLaunchKernelGGL((route_bwd_kernel<float, L, P>), grid, dim3(WG), 0, st, a);
  });
  return hipGetLastError();
}

}  // namespace muon
