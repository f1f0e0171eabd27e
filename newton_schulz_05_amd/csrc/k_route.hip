// Expert router: softmax over the experts, the k largest as choices with
// their gates, the number of choices of every expert, and the balance loss
//   L = coef E sum_e f_e P_e,  f_e = c_e / (k n),  P_e = (1 / n) sum_t p_te
// over the n tokens that have a choice, with gradients through P and the
// gates (the counts c are constants):
//   dp_te = coef E c_e / (k n^2) dL + [e chosen] (gradient of its gate),
//   dlogit = p (dp - sum_e p dp).
// A group of 8 or 16 lanes holds one token's logits in registers, each lane PER
// of them (see expert_of), so the maximum, the sums and the choices are
// reductions over at most 16 lanes, all of them single DPP steps.
#include "ops_dev.hpp"

#include <type_traits>

namespace muon {

namespace {

constexpr int WG = kRouteThreads;

// Order-preserving bits of a float: larger value, larger word; -0 counts as 0.
// Words up to kNone (-inf, an expert that is shut off, and 0, one that is taken)
// are never chosen.
constexpr uint32_t kNone = 0x007fffffu;
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}

// What the choices are made by.  bf16: the 16 bits of the value with the
// expert's complement below them, so that one maximum finds the largest logit
// and the lowest expert that has it.  fp32 has no room for the expert: the
// maximum of the value, then the lowest expert that has it.
template <typename T> struct Choice;
template <> struct Choice<uint16_t> {
  static __device__ __forceinline__ uint32_t key(float v, int expert) {
    return (order_key(v) & 0xffff0000u) | (0xffffu - uint32_t(expert));
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float((k >> 31) ? (k & 0xffff0000u) ^ 0x80000000u : ~(k | 0xffffu));
  }
};
template <> struct Choice<float> {
  static __device__ __forceinline__ uint32_t key(float v, int) { return order_key(v); }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
  }
};

template <int N> __device__ __forceinline__ uint32_t lane_max(uint32_t v) {
  return lane_reduce<N>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int N> __device__ __forceinline__ uint32_t lane_min(uint32_t v) {
  return lane_reduce<N>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

// The i-th expert of lane t: runs of 8 dealt to the lanes in turn, so that a
// group's 16-byte accesses are adjacent (backward of 32768 x 256 fp32 20.9 us,
// 24.8 with PER consecutive experts a lane); fewer than 8 a lane are
// consecutive.  Experts rise with i.
template <int LANES, int PER> __device__ __forceinline__ int expert_of(int t, int i) {
  return PER >= 8 ? ((i >> 3) * LANES + t) * 8 + (i & 7) : t * PER + i;
}

// Takes the largest key left among the group's lanes out of `key`; returns it
// and its expert (a key up to kNone once none is left).
template <typename T, int LANES, int PER>
__device__ __forceinline__ uint32_t take_largest(uint32_t (&key)[PER], int t, int& expert) {
  if constexpr (sizeof(T) == 2) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) best = key[i] > best ? key[i] : best;
    best = lane_max<LANES>(best);
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = key[i] == best ? 0u : key[i];
    expert = 0xffff - int(best & 0xffffu);
    return best;
  } else {
    uint32_t best = key[0], at = 0;
#pragma unroll
    for (int i = 1; i < PER; ++i) {
      at = key[i] > best ? i : at;
      best = key[i] > best ? key[i] : best;
    }
    const uint32_t m = lane_max<LANES>(best);
    expert = int(lane_min<LANES>(best == m ? uint32_t(expert_of<LANES, PER>(t, at)) : 0xffffu));
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = expert == expert_of<LANES, PER>(t, i) ? 0u : key[i];
    return m;
  }
}

// exp(x) for x <= 0 (NaN stays NaN) from the hardware's 2^t: x log2(e) is split
// into its rounded product t and the rest r, and 2^(t + r) = 2^t (1 + r ln 2),
// which keeps the relative error at a few 2^-24 for results down to 2^-126 (x of
// about -87.3); smaller ones are 0.
__device__ __forceinline__ float exp_neg(float x) {
  x = x < -150.0f ? -150.0f : x;  // 2^-216: 0 in fp32
  const float t = x * 1.44269502f;
  const float r = fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269502f, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, r * 0.693147181f, e);
}

// Lane J of every group, in all of the group's lanes.
template <int LANES, int J> __device__ __forceinline__ uint32_t lane_of_group(uint32_t v) {
  const uint32_t lo = dpp<0x150 + J>(v);  // lane J of each 16
  if constexpr (LANES == 16) return lo;
  const uint32_t hi = dpp<0x150 + 8 + J % 8>(v);
  return (threadIdx.x & 8) ? hi : lo;
}

__device__ __forceinline__ float widen(uint16_t x) { return bf2f(x); }
__device__ __forceinline__ float widen(float x) { return x; }
template <typename T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ uint16_t narrow<uint16_t>(float x) { return f2bf(x); }
template <> __device__ __forceinline__ float narrow<float>(float x) { return x; }

// Lane t's PER logits of a token that has `have` of them (0: none are read), as
// stored, by one access for each run that exists whole (at any alignment of an
// element, like load8); floats(): -inf where there is none.
template <typename T, int LANES, int PER> struct Logits {
  typedef T V __attribute__((ext_vector_type(PER < 8 ? PER : 1)));
  typedef T VU __attribute__((ext_vector_type(PER < 8 ? PER : 1), aligned(sizeof(T))));
  Raw8<T> many[PER < 8 ? 1 : PER / 8];
  V few;
  __device__ __forceinline__ void load(const T* row, int t, int have) {
    if constexpr (PER >= 8) {
#pragma unroll
      for (int i = 0; i < PER; i += 8) {
        const int e = expert_of<LANES, PER>(t, i);
        many[i / 8] = load8(row + e, have - e);
      }
    } else {
      const T* p = row + t * PER;
      const int n = have - t * PER;
      if (n >= PER) {
        few = *(const VU*)p;
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) few[i] = i < n ? p[i] : T(0);
      }
    }
  }
  __device__ __forceinline__ void floats(int t, int have, float (&v)[PER]) const {
    if constexpr (PER >= 8) {
#pragma unroll
      for (int i = 0; i < PER; i += 8) {
        float w[8];
        unpack8(many[i / 8], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i + j] = w[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = widen(few[i]);
    }
    if (__ballot(have < LANES * PER)) {  // padding tokens, experts that do not fill the lanes
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = expert_of<LANES, PER>(t, i) < have ? v[i] : -INFINITY;
    }
  }
};

// The loss from x = sum_e c_e (sum_t p_te) over n tokens.
__device__ __forceinline__ void put_loss(const RouteArgs& a, double x, int32_t n) {
  const double tokens = n > 0 ? double(n) : 1.0;
  a.loss[0] = float(double(a.coef) * a.experts * x / (double(a.k) * tokens * tokens));
  a.n_tokens[0] = n;
}
// Counts and mean probability of one expert; returns its c_e (sum_t p_te).
__device__ __forceinline__ double put_expert(const RouteArgs& a, int e, int32_t c, float p, int32_t n) {
  a.counts[e] = c;
  if (a.prob_mean) a.prob_mean[e] = n > 0 ? float(double(p) / n) : 0.0f;
  return double(c) * double(p);
}

// A workgroup takes every gridDim.x-th run of WG / LANES tokens; a lane keeps the
// sums of its experts' probabilities over its tokens, the choices are counted
// in LDS, and both leave one partial sum a workgroup.  A lone workgroup (few
// tokens, see route_parts) finishes the call itself.
template <typename T, int LANES, int PER>
__global__ __launch_bounds__(WG) void route_fwd_kernel(RouteArgs a) {
  constexpr int TOK = WG / LANES, WAVES = WG / 64;
  __shared__ int32_t hist[LANES * PER];
  __shared__ float sums[WAVES][LANES * PER];
  __shared__ int32_t ntok;
  const int t = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  for (int e = threadIdx.x; e < LANES * PER; e += WG) hist[e] = 0;
  if (threadIdx.x == 0) {
    ntok = 0;
    if (blockIdx.x == 0 && gridDim.x > 1) *a.ticket = 0;
  }
  __syncthreads();
  float psum[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) psum[i] = 0.0f;
  int n = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * TOK; row0 < a.rows; row0 += int64_t(gridDim.x) * TOK) {
    const int64_t row = row0 + sub;
    const bool in = row < a.rows;
    const int have = in && (!a.valid || a.valid[row] != 0) ? a.experts : 0;
    Logits<T, LANES, PER> raw;
    raw.load((const T*)a.logits + row * a.ld, t, have);
    float v[PER];
    raw.floats(t, have, v);
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = Choice<T>::key(v[i], expert_of<LANES, PER>(t, i));
    int expert;
    const uint32_t top = take_largest<T, LANES, PER>(key, t, expert);
    uint32_t won = t == 0 ? top : 0u;
    int idx = expert;
    for (int j = 1; j < a.k; ++j) {
      const uint32_t m = take_largest<T, LANES, PER>(key, t, expert);
      won = t == j ? m : won;
      idx = t == j ? expert : idx;
    }
    const bool some = top > kNone, chosen = won > kNone;
    if (!chosen) idx = -1;
    const float mx = some ? Choice<T>::value(top) : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = exp_neg(v[i] - mx);
      s += v[i];
    }
    const float total = lane_sum<LANES>(s);
    const float inv = some ? 1.0f / total : 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) psum[i] = fmaf(v[i], inv, psum[i]);
    float gate = chosen ? exp_neg(Choice<T>::value(won) - mx) * inv : 0.0f;
    if (a.renorm) {
      const float all = lane_sum<LANES>(gate);
      gate = some ? gate / all : 0.0f;
    }
    if (chosen) atomicAdd(&hist[idx], 1);
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
    const float s = across_groups<LANES>(psum[i]);
    if ((threadIdx.x & 63) < LANES) sums[threadIdx.x / 64][expert_of<LANES, PER>(t, i)] = s;
  }
  __syncthreads();
  const bool lone = gridDim.x == 1;
  double x = 0.0;
  for (int e = threadIdx.x; e < a.experts; e += WG) {
    float s = sums[0][e];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += sums[w][e];
    if (lone) {
      x += put_expert(a, e, hist[e], s, ntok);
    } else {
      a.part_p[int64_t(blockIdx.x) * a.experts + e] = s;
      a.part_c[int64_t(blockIdx.x) * a.experts + e] = hist[e];
    }
  }
  if (!lone) {
    if (threadIdx.x == 0) a.part_n[blockIdx.x] = ntok;
    return;
  }
  __shared__ double terms[WAVES];
  for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d, 64);
  if ((threadIdx.x & 63) == 0) terms[threadIdx.x / 64] = x;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < WAVES; ++w) x += terms[w];
    put_loss(a, x, ntok);
  }
}

// Joins the workgroups' sums: 16 experts a workgroup, 64 slices of the at most
// 512 parts, whose at most 8 loads are in flight at once.  The last workgroup
// to finish adds the terms of the loss, in the order of the experts whichever
// it is.
__global__ __launch_bounds__(1024) void route_join_kernel(RouteArgs a) {
  constexpr int SLICES = 64, EACH = kRouteMaxParts / SLICES;
  __shared__ float sp[16][16];
  __shared__ int32_t sc[16][16], sn[16];
  __shared__ int32_t last;
  const int lane = threadIdx.x & 15, slice = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int e = int(blockIdx.x) * 16 + lane;
  float vp[EACH];
  int32_t vc[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int g = slice + SLICES * i;
    const bool have = e < a.experts && g < a.parts;
    vp[i] = have ? a.part_p[int64_t(g) * a.experts + e] : 0.0f;
    vc[i] = have ? a.part_c[int64_t(g) * a.experts + e] : 0;
  }
  int32_t n = int(threadIdx.x) < a.parts ? a.part_n[threadIdx.x] : 0;
  float p = vp[0];
  int32_t c = vc[0];
#pragma unroll
  for (int i = 1; i < EACH; ++i) {
    p += vp[i];
    c += vc[i];
  }
  p = across_groups<16>(p);
  c += __shfl_xor(c, 16, 64);
  c += __shfl_xor(c, 32, 64);
  for (int d = 32; d >= 1; d >>= 1) n += __shfl_xor(n, d, 64);
  if ((threadIdx.x & 63) < 16) {
    sp[wave][lane] = p;
    sc[wave][lane] = c;
  }
  if ((threadIdx.x & 63) == 0) sn[wave] = n;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  n = sn[0];
#pragma unroll
  for (int w = 1; w < 16; ++w) n += sn[w];
  double x = 0.0;
  if (threadIdx.x < 16 && e < a.experts) {
    p = sp[0][lane];
    c = sc[0][lane];
#pragma unroll
    for (int w = 1; w < 16; ++w) {
      p += sp[w][lane];
      c += sc[w][lane];
    }
    x = put_expert(a, e, c, p, n);
  }
  for (int d = 8; d >= 1; d >>= 1) x += __shfl_xor(x, d, 64);
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) {
      __hip_atomic_store(a.terms + blockIdx.x, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
    if (!__shfl(threadIdx.x == 0 ? last : 0, 0, 64)) return;
    x = threadIdx.x < gridDim.x ? __hip_atomic_load(a.terms + threadIdx.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                                : 0.0;
    for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d, 64);
  }
  if (threadIdx.x == 0) put_loss(a, x, n);
}

// A group's lanes are in one wave, whose LDS accesses take place in order; this
// keeps the compiler from moving them.
__device__ __forceinline__ void wave_lds_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// Lane J's choice of every group in turn: dp += its gradient dg at its expert.
// Up to two experts a lane compare; with more, the gradients go through the
// group's own run of LDS, one lane of each group at a time, so that an index
// named more than once is added in the order of the slots (65536 x 128
// bf16, k = 8: 208 instructions a token group by comparison).
template <int LANES, int PER, int J>
__device__ __forceinline__ void add_choices(float (&dp)[PER], float* mem, int t, int idx, float dg, int base, int k) {
  if (J < k) {
    if constexpr (PER <= 2) {
      const int e = int(lane_of_group<LANES, J>(uint32_t(idx))) - base;
      const float x = __uint_as_float(lane_of_group<LANES, J>(__float_as_uint(dg)));
#pragma unroll
      for (int i = 0; i < PER; ++i) dp[i] += e == i ? x : 0.0f;
    } else {
      if (t == J && idx >= 0) atomicAdd(mem + idx, dg);
    }
    if constexpr (J + 1 < LANES) add_choices<LANES, PER, J + 1>(dp, mem, t, idx, dg, base, k);
  }
}

// The value of one of the group's lanes that have one (the largest word, so
// that equals agree on it); the others come with 0.
template <int LANES> __device__ __forceinline__ float reference(float v) {
  return __uint_as_float(lane_max<LANES>(__float_as_uint(v)));
}

template <typename T, int LANES, int PER>
__global__ __launch_bounds__(kRouteBwdThreads) void route_bwd_kernel(RouteBwdArgs a) {
  constexpr int TOK = kRouteBwdThreads / LANES;
  __shared__ __attribute__((aligned(16))) float slots[TOK][PER > 2 ? LANES * PER : 1];
  const int t = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  // one token of a group; the first one's loads are under way while the
  // balance terms, which wait for the counts, are formed
  Logits<T, LANES, PER> raw;
  int have = 0, idx = -1;
  float dg = 0.0f;
  auto fetch = [&](int64_t row) {
    const bool live = row < a.rows && (!a.valid || a.valid[row] != 0);
    have = live ? a.experts : 0;
    raw.load((const T*)a.logits + row * a.ld, t, have);
    // lane t holds the token's choice t
    const bool mine = live && a.dgates && t < a.k;
    idx = mine ? a.idx[row * a.k + t] : -1;
    dg = mine ? a.dgates[row * a.k + t] : 0.0f;
  };
  fetch(int64_t(blockIdx.x) * TOK + sub);
  // A constant added to every dp of a token changes nothing (sum p = 1), so
  // the counts enter as E c_e - sum c, exact in fp64: near balance the
  // differences are what matters.  Counts summed over ranks have a sum beyond
  // 32 bits; it is formed over the lanes in two parts.
  int32_t c[PER];
  uint64_t own = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = expert_of<LANES, PER>(t, i);
    c[i] = e < a.experts ? a.counts[e] : 0;
    own += uint32_t(c[i]);
  }
  auto add = [](uint32_t x, uint32_t y) { return x + y; };
  const double all = 16777216.0 * lane_reduce<LANES>(uint32_t(own >> 24), add) +
                     lane_reduce<LANES>(uint32_t(own) & 0xffffffu, add);
  const int ntok = a.n_tokens[0];
  const double up = ntok > 0 ? double(a.coef) * (a.dloss ? double(a.dloss[0]) : 1.0) / (double(a.k) * ntok * ntok) : 0.0;
  float bal[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) bal[i] = float(up * (double(c[i]) * a.experts - all));
  const int64_t step = int64_t(gridDim.x) * TOK;
  for (int64_t row0 = int64_t(blockIdx.x) * TOK; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + sub;
    const bool in = row < a.rows;
    if (idx < 0 || idx >= a.experts) {
      idx = -1;
      dg = 0.0f;
    }
    float v[PER];
    raw.floats(t, have, v);
    float mx = v[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) mx = fmaxf(mx, v[i]);
    mx = lane_reduce<LANES>(mx, [](float x, float y) { return fmaxf(x, y); });
    const bool some = mx != -INFINITY;
    mx = some ? mx : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = exp_neg(v[i] - mx);
      s += v[i];
    }
    const float total = lane_sum<LANES>(s);
    const float inv = some ? 1.0f / total : 0.0f;
    if (a.dgates && a.renorm) {
      const float q = idx >= 0 ? exp_neg(Elem<T>::load((const T*)a.logits + row * a.ld + idx) - mx) * inv : 0.0f;
      const float sum = lane_sum<LANES>(q);
      const float share = sum > 0.0f ? q / sum : 0.0f;
      // dg - sum share dg by the difference to the gate of the largest share (a
      // lone choice has exactly 0), see below
      const uint32_t most = lane_max<LANES>(__float_as_uint(q));
      dg -= reference<LANES>(idx >= 0 && __float_as_uint(q) == most ? dg : 0.0f);
      const float mid = lane_sum<LANES>(idx >= 0 ? dg * share : 0.0f);
      dg = sum > 0.0f ? (dg - mid) / sum : 0.0f;
    }
    float dp[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) dp[i] = bal[i];
    if (a.dgates) {
      float* mem = slots[sub];
      if constexpr (PER > 2) {
#pragma unroll
        for (int i = 0; i < PER; ++i) mem[expert_of<LANES, PER>(t, i)] = dp[i];
        wave_lds_order();
      }
      add_choices<LANES, PER, 0>(dp, mem, t, idx, dg, t * PER, a.k);
      if constexpr (PER > 2) {
        wave_lds_order();
#pragma unroll
        for (int i = 0; i < PER; ++i) dp[i] = mem[expert_of<LANES, PER>(t, i)];
        wave_lds_order();
      }
    }
    // dlogit = p (dp - sum p dp).  Where one p is near 1 the sum is near its dp
    // and their difference is all roundings, so dp is counted from the most
    // probable expert's (whose exponential is exactly 1): that adds nothing to
    // the sum, and the gradients are sums of the others' small terms.
    float ref = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) ref = v[i] == 1.0f ? dp[i] : ref;
    ref = reference<LANES>(ref);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      dp[i] -= ref;
      dot = fmaf(v[i], dp[i], dot);
    }
    dot = lane_sum<LANES>(dot) * inv;
    const float shift = dot * inv;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] *= fmaf(dp[i], inv, -shift);
    if (__ballot(!some)) {  // 0 by selection: what reaches a token may not be finite
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = some ? v[i] : 0.0f;
    }
    if (in) {
      T* out = (T*)a.dlogits + row * a.ld_d;
      if constexpr (PER >= 8) {
#pragma unroll
        for (int i = 0; i < PER; i += 8) {
          const int e = expert_of<LANES, PER>(t, i);
          float w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = v[i + j];
          store8(out + e, a.experts - e, pack8(w, (const T*)nullptr));
        }
      } else if (t * PER + PER <= a.experts) {
        typename Logits<T, LANES, PER>::V w;
#pragma unroll
        for (int i = 0; i < PER; ++i) w[i] = narrow<T>(v[i]);
        *(typename Logits<T, LANES, PER>::VU*)(out + t * PER) = w;
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (t * PER + i < a.experts) Elem<T>::store(out + t * PER + i, v[i]);
      }
    }
    fetch(row + step);
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
  by_experts(a.experts, [&](auto lanes, auto per) {
    constexpr int L = decltype(lanes)::value, P = decltype(per)::value;
    if (bf16) hipLaunchKernelGGL((route_fwd_kernel<uint16_t, L, P>), dim3(unsigned(a.parts)), dim3(WG), 0, st, a);
    else hipLaunchKernelGGL((route_fwd_kernel<float, L, P>), dim3(unsigned(a.parts)), dim3(WG), 0, st, a);
  });
  if (a.parts > 1)
    hipLaunchKernelGGL(route_join_kernel, dim3(unsigned((a.experts + 15) / 16)), dim3(1024), 0, st, a);
  return hipGetLastError();
}

hipError_t run_route_bwd(const RouteBwdArgs& a, bool bf16, hipStream_t st) {
  by_experts(a.experts, [&](auto lanes, auto per) {
    constexpr int L = decltype(lanes)::value, P = decltype(per)::value;
    const int64_t need = (a.rows + kRouteBwdThreads / L - 1) / (kRouteBwdThreads / L);
    const dim3 grid(unsigned(std::min<int64_t>(need, 1024)));
    if (bf16) hipLaunchKernelGGL((route_bwd_kernel<uint16_t, L, P>), grid, dim3(kRouteBwdThreads), 0, st, a);
    else hipLaunchKernelGGL((route_bwd_kernel<float, L, P>), grid, dim3(kRouteBwdThreads), 0, st, a);
  });
  return hipGetLastError();
}

}  // namespace muon
