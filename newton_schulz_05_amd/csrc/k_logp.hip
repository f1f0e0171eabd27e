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

// NT threads take a row, or with a.parts > 1 every a.parts-th run of pieces of
// it; U pieces a thread are in flight at once.  One pass: every piece raises the
// thread's maximum first and then adds its terms, so that the old sum is scaled
// once for 4 or 8 elements.  Long rows are bound by memory: 8192 x 65536 bf16
// 162 us, 6.6 TB/s; two thirds of the cycles are instructions, of which the exponential is
// the largest part (8.5 an element, it counts four).
template <typename T, int NT, int WG, int U, bool STREAM>
__global__ __launch_bounds__(WG) void logp_fwd_kernel(LogpArgs a) {
  constexpr int ROWS = WG / NT, NW = NT / 64, N = Piece<T>::N;
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
    if (some) {  // a row without a target is not read
      const int cols = int(a.cols), at = int(target);
      for (int col0 = part * NT * N * U; col0 < cols; col0 += a.parts * NT * N * U) {
        Piece<T> raw[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int col = col0 + (i * NT + t) * N;
          raw[i].template load<STREAM>(x + col, cols - col);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int col = col0 + (i * NT + t) * N;
          float v[N];
          raw[i].get(v);
          if (col + N > cols || unsigned(at - col) < unsigned(N)) {
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = col + j < cols && col + j != at ? v[j] : -INFINITY;
          }
          add_block(mine, v, c);
        }
      }
    }
    mine = lanes_join<64>(mine, c);
    if constexpr (NW > 1) {
      const int first = threadIdx.x / NT * NW;
      __syncthreads();
      if (threadIdx.x % 64 == 0) waves[threadIdx.x / 64] = mine;
      __syncthreads();
      mine = waves[first];
#pragma unroll
      for (int w = 1; w < NW; ++w) mine = join(mine, waves[first + w], c);
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

// Many short rows: LANES lanes take K of them at once, whole (cols <= LANES U
// pieces), and finish them together, a lane a row: the logarithms of one row cost a
// wave as much as those of 64, and half of a row of 500.  Rows without a target are
// read here, their values are not used.
template <typename T, int LANES, int U, int K>
__global__ __launch_bounds__(256) void logp_short_kernel(LogpArgs a) {
  constexpr int N = Piece<T>::N, GROUPS = 256 / LANES;
  const int t = threadIdx.x % LANES, cols = int(a.cols);
  const int64_t step = int64_t(gridDim.x) * (GROUPS * K);
  for (int64_t first = int64_t(blockIdx.x) * (GROUPS * K); first < a.rows; first += step) {
    const int64_t row0 = first + threadIdx.x / LANES * K;
    // lane k of a group looks after row k
    const int64_t own = row0 + (t < K ? t : 0);
    const int64_t target = t < K && own < a.rows ? a.targets[own] : -1;
    const bool some = uint64_t(target) < uint64_t(a.cols);
    const int at = some ? int(target) : -1;
    const float xt = some ? Elem<T>::load((const T*)a.logits + own * a.ld + at) : 0.0f;
    Piece<T> raw[K][U];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int col = (i * LANES + t) * N;
        const bool in = row0 + k < a.rows;
        raw[k][i].template load<false>((const T*)a.logits + (in ? row0 + k : 0) * a.ld + col, in ? cols - col : 0);
      }
    MaxSum mine{-INFINITY, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int hit = __shfl(at, (threadIdx.x & 63) / LANES * LANES + k, 64);
      float v[U * N];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float w[N];
        raw[k][i].get(w);
        const int col = (i * LANES + t) * N;
#pragma unroll
        for (int j = 0; j < N; ++j) v[i * N + j] = w[j];
        if (col + N > cols || unsigned(hit - col) < unsigned(N)) {
#pragma unroll
          for (int j = 0; j < N; ++j) v[i * N + j] = col + j < cols && col + j != hit ? w[j] : -INFINITY;
        }
      }
      float m = v[0];
#pragma unroll
      for (int j = 1; j < U * N; ++j) m = fmaxf(m, v[j]);
      m = lane_reduce<LANES>(m, [](float x, float y) { return fmaxf(x, y); });
      const float r = above(m);
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < U * N; ++j) s += grow(v[j], r, a.scale2);
      s = lane_sum<LANES>(s);
      if (t == k) mine = {m, s};
    }
    if (t < K && own < a.rows) put_row(a, own, mine, some, xt);
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

// Maximum and sum of a row's terms by the NT threads that share it, the target's
// own among them.  Every thread has the result, and has read all that it reads
// before any of them leaves.
template <typename T, int NT> __device__ __forceinline__ MaxSum row_sum(const T* x, int cols, int t, float c, MaxSum* waves) {
  constexpr int N = Piece<T>::N, NW = NT / 64;
  MaxSum mine{-INFINITY, 0.0f};
#pragma unroll 1
  for (int col = t * N; col < cols; col += NT * N) {
    Piece<T> raw;
    raw.template load<false>(x + col, cols - col);
    float v[N];
    raw.get(v);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = col + j < cols ? v[j] : -INFINITY;
    add_block(mine, v, c);
  }
  mine = lanes_join<(NT < 64 ? NT : 64)>(mine, c);
  if constexpr (NW > 1) {
    __syncthreads();
    if (threadIdx.x % 64 == 0) waves[threadIdx.x / 64] = mine;
    __syncthreads();
    mine = waves[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) mine = join(mine, waves[w], c);
  }
  return mine;
}

// One run of a row's gradient: U pieces of every thread from col0 on, of a
// probability exp(scale (x_j - off) + base) each.  off counts where SHIFT says so.
template <bool SHIFT, int STEP, typename T, int U, bool STREAM>
__device__ __forceinline__ void put_gradient(const LogpBwdArgs& a, int64_t row, int col0, int at, float g, float off,
                                             float base) {
  constexpr int N = Piece<T>::N;
  const int cols = int(a.cols);
  const T* x = (const T*)a.logits + row * a.ld;
  T* out = (T*)a.dlogits + row * a.ld_d;
  Piece<T> raw[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int col = col0 + i * STEP;
    raw[i].template load<STREAM>(x + col, cols - col);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int col = col0 + i * STEP;
    float v[N];
    raw[i].get(v);
#pragma unroll
    for (int j = 0; j < N; ++j)
      v[j] = -g * __builtin_amdgcn_exp2f(fmaf(SHIFT ? v[j] - off : v[j], a.scale, base) * 1.44269504f);
    if (unsigned(at - col) < unsigned(N)) {
      const float own = -g * expm1f(a.logp[row]);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = col + j == at ? own : v[j];
    }
    Piece<T>::store(out + col, cols - col, v, a.stream_out);
  }
}
template <int STEP, typename T, int U>
__device__ __forceinline__ void put_zeros(const LogpBwdArgs& a, int64_t row, int col0) {
  const int cols = int(a.cols);
  T* out = (T*)a.dlogits + row * a.ld_d;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int col = col0 + i * STEP;
    const float zero[Piece<T>::N] = {};
    Piece<T>::store(out + col, cols - col, zero, a.stream_out);
  }
}

// A statistic of at most this size, rounded to fp32, leaves a probability within
// 2^-19 of itself.
constexpr float kNear = 64.0f;

// NT threads take U NT pieces of a row; blockIdx.x counts these along it,
// blockIdx.y the rows.  Bound by memory: 8192 x 65536 bf16, a tenth of the rows
// without a target, 331 us, 6.2 TB/s; rows at odd addresses (4096 x 65521) 212 us, 5.1.
//
// A probability is exp(z_j - lse) as long as lse is small.  A large one has lost what
// it adds to the row's maximum (all of it at the lowest value, where it cannot hold
// the logarithm of the vocabulary): the target's logit and logp take its place, which
// an offset of the whole row does not change, or, where logp is large too, the row's
// maximum and sum, formed again.  The latter is done for the whole row by the
// threads of one blockIdx.x, and so is a row whose target's logit may be overwritten
// while others still read it (dlogits in the logits' place).  Which one goes by a hash
// of the row: row % gridDim.x leaves most compute units without such rows (8192 x
// 65536 bf16, all rows at 1000, into another tensor 325 us; in place 385, 730 by
// row % gridDim.x, 1490 by blockIdx.x 0; with unlikely targets as well 443).
template <typename T, int NT, int WG, int U, bool STREAM>
__global__ __launch_bounds__(WG, U == 1 ? 8 : 1) void logp_bwd_kernel(LogpBwdArgs a) {
  constexpr int ROWS = WG / NT, N = Piece<T>::N, STEP = NT * N, RUN = STEP * U;
  static_assert(NT <= 64 || ROWS == 1);  // the barriers below are a row's
  __shared__ MaxSum waves[WG / 64];
  const int t = threadIdx.x % NT;
  for (int64_t row = int64_t(blockIdx.y) * ROWS + threadIdx.x / NT; row < a.rows; row += int64_t(gridDim.y) * ROWS) {
    const int64_t target = a.targets[row];
    const float lse = a.lse[row], up = a.dlogp[row], g = up * a.scale;
    const int at = int(target);
    bool some = uint64_t(target) < uint64_t(a.cols) && up != 0.0f, whole = false;
    float off = 0.0f, base = -lse;
    if (some && fabsf(lse) <= kNear) {
      // short rows are bound by instructions: a way without the subtraction, in the
      // registers of eight waves a SIMD (30000 x 500 bf16 13.9 us, 15.2 without the
      // former, 15.0 without the latter)
      if constexpr (U == 1) {
        put_gradient<false, STEP, T, U, STREAM>(a, row, int(blockIdx.x) * RUN + t * N, at, g, off, base);
        continue;
      }
    } else if (some) {
      const T* x = (const T*)a.logits + row * a.ld;
      const float logp = a.logp[row];
      const bool near = fabsf(logp) <= kNear;
      whole = !near || a.in_place;
      if (whole && blockIdx.x != (uint32_t(row) * 2654435761u >> 16) % gridDim.x) continue;
      if (near) {
        off = Elem<T>::load(x + target);
        base = logp;
        some = off != -INFINITY;  // else the row is -inf throughout
        if constexpr (NT > 64) {
          asm volatile("" ::"v"(off));  // the load has returned
          __syncthreads();
        }
      } else {
        const MaxSum m = row_sum<T, NT>(x, int(a.cols), t, a.scale2, waves);
        off = above(m.m);
        base = -logf(m.s);
        some = m.s != 0.0f;
      }
    }
    const int from = whole ? 0 : int(blockIdx.x) * RUN, to = whole ? int(a.cols) : from + 1;
#pragma unroll 1
    for (int run = from; run < to; run += RUN) {
      if (some) put_gradient<true, STEP, T, U, STREAM>(a, row, run + t * N, at, g, off, base);
      else put_zeros<STEP, T, U>(a, row, run + t * N);
    }
  }
}

template <int V> using Num = std::integral_constant<int, V>;
template <bool V> using Flag = std::integral_constant<bool, V>;

}  // namespace

hipError_t run_logp_fwd(const LogpArgs& a, bool bf16, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  auto go = [&](auto t, auto nt, auto u, auto stream) {
    constexpr int NT = decltype(nt)::value, WG = NT > 256 ? NT : 256;
    const int64_t groups = (a.rows + WG / NT - 1) / (WG / NT);
    hipLaunchKernelGGL((logp_fwd_kernel<decltype(t), NT, WG, decltype(u)::value, decltype(stream)::value>),
                       dim3(unsigned(std::min(groups, kOpsMaxGrid) * a.parts)), dim3(WG), 0, st, a);
  };
  auto shorts = [&](auto t, auto l, auto u, auto k) {
    constexpr int L = decltype(l)::value, U = decltype(u)::value, K = decltype(k)::value, EACH = 256 / L * K;
    const int64_t groups = (a.rows + EACH - 1) / EACH;
    hipLaunchKernelGGL((logp_short_kernel<decltype(t), L, U, K>), dim3(unsigned(std::min(groups, kOpsMaxGrid))), dim3(256), 0,
                       st, a);
  };
  auto by_cols = [&](auto t) {
    // A wave a row where rows are short or there are many of them: what lanes and
    // pieces behind a row's end cost, and a workgroup's barriers, are most of it
    // there (30000 x 500 bf16 18.8 us, 34.6 with two waves a row of two pieces,
    // 61.0 with four; 8192 x 5000 19.0, 22.5, 28.2; 16384 x 2000 fp32 30.1, 28.4,
    // 32.0; but 600 x 5000 6.3, 5.7, 5.5).  Longer rows: four waves of four pieces
    // (4096 x 32768 bf16 54.0 us, 57.5 with a wave; 4096 x 131072 171 and 180), or
    // eight where there are few of them (1 x 32768 4.8 us with eight, 4.9 with
    // sixteen; 300 x 32768 8.8 and 10.2; 300 x 5000, of 625 pieces, 5.8 and 4.6 with
    // four).
    constexpr int N = Piece<decltype(t)>::N;
    const bool many = a.rows >= 4096;
    if (a.rows >= 4096 && a.cols <= 32 * N) {
      // 60000 x 100 bf16 8.8 us, 19.3 with 64 lanes a row; 60000 x 256 10.4 and 18.2
      a.cols <= 16 * N ? shorts(t, Num<16>{}, Num<1>{}, Num<4>{}) : shorts(t, Num<16>{}, Num<2>{}, Num<2>{});
    } else if (a.rows >= 16384 && a.cols <= 128 * N) {
      // 30000 x 500 bf16 12.1 us, 18.7 with a wave for each row, 13.7 with a wave for
      // four; 32768 x 1000 17.3 and 23.2; but 8192 x 1000 7.8 and 7.6 with a wave for
      // each, 5000 x 500 6.7 and 5.0.
      a.cols <= 64 * N ? shorts(t, Num<16>{}, Num<4>{}, Num<2>{}) : shorts(t, Num<64>{}, Num<2>{}, Num<2>{});
    } else if (a.cols <= 64 * N || (a.cols <= 2048 && !many)) go(t, Num<64>{}, Num<1>{}, Flag<false>{});
    else if (a.cols <= 1024 * N && many) go(t, Num<64>{}, Num<2>{}, Flag<false>{});
    else if (a.cols > 1024 * N && a.rows < kLogpFewRows && a.parts == 1) go(t, Num<512>{}, Num<4>{}, Flag<false>{});
    else if (a.rows * a.cols * int64_t(sizeof(t)) > kStreamIn) go(t, Num<256>{}, Num<4>{}, Flag<true>{});
    else go(t, Num<256>{}, Num<4>{}, Flag<false>{});
  };
  bf16 ? by_cols(uint16_t{}) : by_cols(float{});
  if (a.parts > 1) hipLaunchKernelGGL(logp_join_kernel, dim3(unsigned(a.rows)), dim3(64), 0, st, a, bf16);
  return hipGetLastError();
}

hipError_t run_logp_bwd(const LogpBwdArgs& args, bool bf16, hipStream_t st) {
  LogpBwdArgs a = args;
  a.stream_out = a.rows * a.cols * (bf16 ? 2 : 4) > kStreamOut;
  a.in_place = a.dlogits == a.logits;
  auto go = [&](auto t, auto nt, auto u, auto stream) {
    constexpr int NT = decltype(nt)::value, WG = 256, U = decltype(u)::value, RUN = NT * Piece<decltype(t)>::N * U;
    const int64_t runs = (a.cols + RUN - 1) / RUN, groups = (a.rows + WG / NT - 1) / (WG / NT);
    hipLaunchKernelGGL((logp_bwd_kernel<decltype(t), NT, WG, U, decltype(stream)::value>),
                       dim3(unsigned(runs), unsigned(std::min<int64_t>(groups, 65535))), dim3(WG), 0, st, a);
  };
  auto by_cols = [&](auto t) {
    // The fewest lanes that hold a row of up to 32 pieces: 60000 x 100 bf16 8.8 us, 19.7
    // with 64 lanes; 60000 x 256 12.9 and 19.1.  Two and four rows a lane at once:
    // no gain.
    constexpr int N = Piece<decltype(t)>::N;
    if (a.cols <= 16 * N) go(t, Num<16>{}, Num<1>{}, Flag<false>{});
    else if (a.cols <= 32 * N) go(t, Num<32>{}, Num<1>{}, Flag<false>{});
    else if (a.cols <= 256 * N) go(t, Num<64>{}, Num<1>{}, Flag<false>{});
    else if (a.rows * a.cols * int64_t(sizeof(t)) > kStreamIn) go(t, Num<256>{}, Num<4>{}, Flag<true>{});
    else go(t, Num<256>{}, Num<4>{}, Flag<false>{});
  };
  bf16 ? by_cols(uint16_t{}) : by_cols(float{});
  return hipGetLastError();
}

}  // namespace muon
