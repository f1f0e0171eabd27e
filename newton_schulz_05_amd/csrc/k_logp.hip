// Log-probabilities of the tokens' targets, and their gradient:
//
//   forward   z = scale x, lse = log sum_j exp z_j, logp = z_t - lse
//   backward  dx_j = scale dlogp ([j = t] - exp(z_j - lse))
//
// The forward pass reads a row once with a running maximum and sum in every
// thread.  The target's own term stays out of the sums: with e = exp(z_t - M) and
// the others' sum s, logp = -log(1 + s / e), which keeps its relative accuracy
// where the target is nearly certain and s is far below the last place of 1.
#include "ops_dev.hpp"

#include <type_traits>

namespace muon {

namespace {

// Maximum m and sum s of exp2((x - m) c) over what a thread, then a row, has.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ float above(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ float grow(float x, float m, float c) { return __builtin_amdgcn_exp2f((x - m) * c); }

// Both parts over one maximum.
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
  const float m = fmaxf(a.m, b.m), r = above(m);
  return {m, fmaf(a.s, grow(a.m, r, c), b.s * grow(b.m, r, c))};
}

template <int N> __device__ __forceinline__ MaxSum lanes_join(MaxSum a, float c) {
  const float m = lane_reduce<N>(a.m, [](float x, float y) { return fmaxf(x, y); });
  return {m, lane_sum<N>(a.s * grow(a.m, above(m), c))};
}

// Adds N elements.
template <int N> __device__ __forceinline__ void add_block(MaxSum& a, const float (&v)[N], float c) {
  float m = a.m;
#pragma unroll
  for (int j = 0; j < N; ++j) m = fmaxf(m, v[j]);
  const float r = above(m);
  float s = a.s * grow(a.m, r, c);
#pragma unroll
  for (int j = 0; j < N; ++j) s += grow(v[j], r, c);
  a = {m, s};
}

// logp and lse of a row from the others' maximum and sum and the target's logit.
__device__ __forceinline__ void put_row(const LogpArgs& a, int64_t row, MaxSum rest, bool some, float xt) {
  float logp = 0.0f, lse = 0.0f;
  if (some) {
    const float m = fmaxf(rest.m, xt), r = above(m);
    const float d = (xt - r) * a.scale, e = expf(d), s = rest.s * grow(rest.m, r, a.scale2);
    lse = fmaf(r, a.scale, logf(e + s));
    const float ratio = s / e;
    logp = ratio < 1.0f ? -log1pf(ratio) : d - logf(e + s);
    if (e + s == 0.0f) logp = 0.0f;  // no word is possible: lse = -inf
  }
  a.logp[row] = logp;
  a.lse[row] = lse;
}

// NT threads take a row, or with a.parts > 1 every a.parts-th run of vectors of
// it; U vectors of 8 elements a thread are in flight at once.
template <typename T, int NT, int WG, int U>
__global__ __launch_bounds__(WG) void logp_fwd_kernel(LogpArgs a) {
  constexpr int ROWS = WG / NT, NW = NT / 64;
  __shared__ MaxSum waves[WG / 64];
  const int t = threadIdx.x % NT;
  const int part = int(blockIdx.x) % a.parts;
  const int64_t group = int64_t(blockIdx.x) / a.parts, groups = gridDim.x / a.parts;
  const float c = a.scale2;
  for (int64_t row0 = group * ROWS; row0 < a.rows; row0 += groups * ROWS) {
    const int64_t row = row0 + threadIdx.x / NT;
    const bool live = row < a.rows;
    const int64_t target = live ? a.targets[row] : -1;
    const bool some = uint64_t(target) < uint64_t(a.cols);
    const T* x = (const T*)a.logits + (live ? row : 0) * a.ld;
    const float xt = some ? Elem<T>::load(x + target) : 0.0f;
    MaxSum mine{-INFINITY, 0.0f};
    if (some) {
      const int cols = int(a.cols), at = int(target);
      for (int col0 = part * NT * 8 * U; col0 < cols; col0 += a.parts * NT * 8 * U) {
        Raw8<T> raw[U];
        float v[U][8];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int col = col0 + (i * NT + t) * 8;
          raw[i] = load8(x + col, cols - col);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int col = col0 + (i * NT + t) * 8;
          unpack8(raw[i], v[i]);
          if (col + 8 > cols || unsigned(at - col) < 8u) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = col + j < cols && col + j != at ? v[i][j] : -INFINITY;
          }
          add_block(mine, v[i], c);
        }
      }
    }
    mine = lanes_join<64>(mine, c);
    if constexpr (NW > 1) {
      __syncthreads();
      if (threadIdx.x % 64 == 0) waves[threadIdx.x / 64] = mine;
      __syncthreads();
      mine = waves[threadIdx.x / NT * NW];
#pragma unroll
      for (int w = 1; w < NW; ++w) mine = join(mine, waves[threadIdx.x / NT * NW + w], c);
    }
    if (t == 0 && live) {
      if (a.parts == 1) {
        put_row(a, row, mine, some, xt);
      } else {
        float* to = a.part + (row * a.parts + part) * 2;
        to[0] = mine.m;
        to[1] = mine.s;
      }
    }
  }
}

// Joins the parts of a row, one a lane.
__global__ __launch_bounds__(64) void logp_join_kernel(LogpArgs a, bool bf16) {
  static_assert(kLogpMaxParts == 64);
  const int64_t row = blockIdx.x;
  const int64_t target = a.targets[row];
  const bool some = uint64_t(target) < uint64_t(a.cols);
  const int64_t at = row * a.ld + target;
  const float xt = !some ? 0.0f : bf16 ? bf2f(((const uint16_t*)a.logits)[at]) : ((const float*)a.logits)[at];
  const int lane = threadIdx.x;
  MaxSum mine{-INFINITY, 0.0f};
  if (lane < a.parts) {
    const float* from = a.part + (row * a.parts + lane) * 2;
    mine = {from[0], from[1]};
  }
  mine = lanes_join<64>(mine, a.scale2);
  if (lane == 0) put_row(a, row, mine, some, xt);
}

// NT threads take 8 U NT elements of a row; blockIdx.x counts these along it,
// blockIdx.y the rows.
template <typename T, int NT, int WG, int U>
__global__ __launch_bounds__(WG) void logp_bwd_kernel(LogpBwdArgs a) {
  constexpr int ROWS = WG / NT;
  const int t = threadIdx.x % NT;
  const int cols = int(a.cols), col0 = int(blockIdx.x) * (NT * 8 * U) + t * 8;
  for (int64_t row = int64_t(blockIdx.y) * ROWS + threadIdx.x / NT; row < a.rows; row += int64_t(gridDim.y) * ROWS) {
    const int64_t target = a.targets[row];
    const float lse = a.lse[row], g = a.dlogp[row] * a.scale;
    const bool some = uint64_t(target) < uint64_t(a.cols) && a.dlogp[row] != 0.0f && lse != -INFINITY;
    const T* x = (const T*)a.logits + row * a.ld;
    T* out = (T*)a.dlogits + row * a.ld_d;
    if (!some) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int col = col0 + i * NT * 8;
        const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        store8(out + col, cols - col, pack8(zero, (const T*)nullptr));
      }
      continue;
    }
    Raw8<T> raw[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int col = col0 + i * NT * 8;
      raw[i] = load8(x + col, cols - col);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int col = col0 + i * NT * 8;
      float v[8];
      unpack8(raw[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = -g * __builtin_amdgcn_exp2f(fmaf(v[j], a.scale, -lse) * 1.44269504f);
      if (uint64_t(target - col) < 8) {
        const float own = -g * expm1f(a.logp[row]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = col + j == target ? own : v[j];
      }
      store8(out + col, cols - col, pack8(v, (const T*)nullptr));
    }
  }
}

}  // namespace

hipError_t run_logp_fwd(const LogpArgs& a, bool bf16, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  auto go = [&](auto t, auto nt, auto wg, auto u) {
    constexpr int NT = decltype(nt)::value, WG = decltype(wg)::value;
    const int64_t groups = (a.rows + WG / NT - 1) / (WG / NT);
    hipLaunchKernelGGL((logp_fwd_kernel<decltype(t), NT, WG, decltype(u)::value>),
                       dim3(unsigned(std::min(groups, kOpsMaxGrid) * a.parts)), dim3(WG), 0, st, a);
  };
  auto by_cols = [&](auto t) {
    typedef std::integral_constant<int, 64> I64;
    typedef std::integral_constant<int, 256> I256;
    if (a.cols <= 2048) go(t, I64{}, I256{}, std::integral_constant<int, 1>{});
    else go(t, I256{}, I256{}, std::integral_constant<int, 4>{});
  };
  bf16 ? by_cols(uint16_t{}) : by_cols(float{});
  if (a.parts > 1) hipLaunchKernelGGL(logp_join_kernel, dim3(unsigned(a.rows)), dim3(64), 0, st, a, bf16);
  return hipGetLastError();
}

hipError_t run_logp_bwd(const LogpBwdArgs& a, bool bf16, hipStream_t st) {
  auto go = [&](auto t, auto nt, auto wg, auto u) {
    constexpr int NT = decltype(nt)::value, WG = decltype(wg)::value, U = decltype(u)::value;
    const int64_t runs = (a.cols + NT * 8 * U - 1) / (NT * 8 * U), groups = (a.rows + WG / NT - 1) / (WG / NT);
    hipLaunchKernelGGL((logp_bwd_kernel<decltype(t), NT, WG, U>), dim3(unsigned(runs), unsigned(std::min<int64_t>(groups, 65535))),
                       dim3(WG), 0, st, a);
  };
  auto by_cols = [&](auto t) {
    typedef std::integral_constant<int, 64> I64;
    typedef std::integral_constant<int, 256> I256;
    if (a.cols <= 2048) go(t, I64{}, I256{}, std::integral_constant<int, 1>{});
    else go(t, I256{}, I256{}, std::integral_constant<int, 4>{});
  };
  bf16 ? by_cols(uint16_t{}) : by_cols(float{});
  return hipGetLastError();
}

}  // namespace muon
