// Norm of every query and key head with the position rotation, forward and
// backward:
//
//   forward   r = 1 / sqrt(mean(x^2) + eps), y = x r gamma, and in the first
//             rot elements every pair (a, b) turned by the token's angle,
//             (a c - b s, b c + a s)
//   backward  g = dy turned back, dgamma = sum over rows of g x r,
//             dx = r (g gamma - x r mean(g gamma x r))
//
// A head's row is read once and held by 4 to 64 lanes, 16 elements each.  Both
// elements of a pair are one lane's, so turning needs no exchange between lanes.
// Sums are fp32; each output is rounded once.
#include "ops_dev.hpp"

#include <type_traits>

// Products and sums are joined only where fmaf says so, so that every variant
// rounds alike.
#pragma clang fp contract(off)

namespace muon {

namespace {

constexpr int WG = kHeadThreads;

__device__ __forceinline__ uint32_t quotient(uint32_t r, const FastDiv& f) {
  return f.d == 1 ? r : __umulhi(r, f.mul) >> f.shift;
}

// What does not fill its pieces: nothing; the angles alone (interleaved pairs,
// rot no multiple of a piece); elements as well.  The last piece of a segment then
// begins so early that it is whole: the elements that two lanes hold are written
// by both, the same bits, and enter the sums once.  (Pieces with elements missing,
// which segments shorter than a piece leave, take three times the instructions:
// 2 x 4096 tokens of 24 + 8 heads of 90 bf16 50 us forward with them, 38 so.)
enum Ragged { kWhole, kRaggedAngles, kOverlap, kRagged };
constexpr bool ragged_angles(int rag, bool inter) {
  return rag == kRaggedAngles || rag == kRagged || (rag == kOverlap && inter);
}

// What a lane holds of every row: 16 elements in pieces of 16 bytes, n[i] of
// them at column c[i], the first skip[i] of which another lane counts.  A
// segment's pieces are dealt to its lanes in turn, so that a wave's accesses are
// adjacent in either type.
template <typename T> struct LanePart {
  static constexpr int E = Piece<T>::N, P = 16 / E;
  int c[P], n[P], skip[P];
  bool turned;
};
__device__ __forceinline__ int some(int n, int most) { return n < 0 ? 0 : n > most ? most : n; }

template <int RAG, typename T, bool INTER> __device__ __forceinline__ LanePart<T> lane_part(int t, int dim, int rot) {
  constexpr int E = LanePart<T>::E, P = LanePart<T>::P;
  LanePart<T> p;
  const int half = rot / 2, first = INTER ? 0 : (half + 7) / 8;
  p.turned = INTER || t < first;
  if (INTER || t >= first) {
    const int from = INTER ? 0 : rot, lanes = (dim - from + 15) / 16, u = t - first;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      p.c[i] = from + E * (u + lanes * i);
      p.n[i] = u < lanes ? some(dim - p.c[i], E) : 0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      p.c[i] = E * (t + first * i);
      p.c[P / 2 + i] = half + p.c[i];
      p.n[i] = p.n[P / 2 + i] = some(half - p.c[i], E);
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    p.skip[i] = RAG == kOverlap && p.n[i] > 0 ? E - p.n[i] : 0;
    p.c[i] -= p.skip[i];
    p.n[i] += p.skip[i];
  }
  return p;
}

// A lane's elements of a row.
template <typename T> struct Held {
  Piece<T> r[LanePart<T>::P];
};
template <int RAG, typename T>
__device__ __forceinline__ void load_held(const T* row, const LanePart<T>& p, bool live, int dim, Held<T>& h) {
#pragma unroll
  for (int i = 0; i < LanePart<T>::P; ++i) {
    const int n = live ? p.n[i] : 0;
    if constexpr (RAG == kRagged && sizeof(T) == 2)
      h.r[i].r = load_row8(row, unsigned(p.c[i]), n > 0 ? dim - p.c[i] : 0, dim);
    else h.r[i].template load<false>(row + p.c[i], RAG == kRagged ? n : (n > 0 ? LanePart<T>::E : 0));
  }
}
template <int RAG, typename T>
__device__ __forceinline__ void unpack_held(Held<T> h, const LanePart<T>& p, bool live, int dim, float (&v)[16]) {
  constexpr int E = LanePart<T>::E;
#pragma unroll
  for (int i = 0; i < LanePart<T>::P; ++i) {
    const int n = live ? p.n[i] : 0;
    if constexpr (RAG == kRagged && sizeof(T) == 2) settle8(h.r[i].r, n > 0 ? dim - p.c[i] : 0, dim);
    float w[E];
    h.r[i].get(w);
#pragma unroll
    for (int j = 0; j < E; ++j) v[E * i + j] = RAG != kRagged || j < n ? w[j] : 0.0f;
  }
}
// Whether another lane counts element j; the elements that this lane counts, 0 for
// the others, infinite ones too.
template <int RAG, typename T> __device__ __forceinline__ bool skipped(const LanePart<T>& p, int j) {
  return RAG == kOverlap && j % LanePart<T>::E < p.skip[j / LanePart<T>::E];
}
template <int RAG, typename T>
__device__ __forceinline__ void counted(const LanePart<T>& p, const float (&v)[16], float (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = skipped<RAG>(p, j) ? 0.0f : v[j];
}
template <int RAG, typename T>
__device__ __forceinline__ void store_held(T* row, const LanePart<T>& p, bool live, const float (&v)[16], bool stream) {
  constexpr int E = LanePart<T>::E;
#pragma unroll
  for (int i = 0; i < LanePart<T>::P; ++i) {
    const int n = live ? p.n[i] : 0;
    float w[E];
#pragma unroll
    for (int j = 0; j < E; ++j) w[j] = v[E * i + j];
    Piece<T>::store(row + p.c[i], RAG == kRagged ? n : (n > 0 ? E : 0), w, stream);
  }
}

// gamma, in fp32 whatever it is stored in; 1 if null.  Ragged pieces are read
// like those of a row of dim.
template <int RAG, int E, typename W>
__device__ __forceinline__ void load_gamma(const W* gamma, int col, int n, int dim, float* v) {
  float w[8];
  Raw8<W> r;
  if constexpr (RAG == kRagged) {
    r = load_row8(gamma, unsigned(col), n > 0 ? dim - col : 0, dim);
    settle8(r, n > 0 ? dim - col : 0, dim);
  } else {
    r = load8(gamma + col, n > 0 ? E : 0);
  }
  unpack8(r, w);
#pragma unroll
  for (int j = 0; j < E; ++j) v[j] = w[j];
}
template <int RAG, typename T>
__device__ __forceinline__ void load_gamma(const void* gamma, bool bf16, const LanePart<T>& p, int dim, float (&v)[16]) {
  constexpr int E = LanePart<T>::E;
#pragma unroll
  for (int i = 0; i < LanePart<T>::P; ++i) {
    if (!gamma) {
#pragma unroll
      for (int j = 0; j < E; ++j) v[E * i + j] = 1.0f;
    } else if (bf16) {
      load_gamma<RAG, E>((const uint16_t*)gamma, p.c[i], p.n[i], dim, v + E * i);
    } else {
      load_gamma<RAG, E>((const float*)gamma, p.c[i], p.n[i], dim, v + E * i);
    }
  }
}

// N consecutive angles at p, of which n exist.
template <int N> __device__ __forceinline__ void load_run(const float* p, int n, float* v) {
  if constexpr (N == 2) {
    if (n >= 2) {
      const f32x2 w = *(const f32x2_u*)p;
      v[0] = w[0];
      v[1] = w[1];
    } else {
      v[0] = n > 0 ? *p : 0.0f;
      v[1] = 0.0f;
    }
  } else if constexpr (N == 4) {
    Piece<float> w;
    float u[4];
    w.load<false>(p, n);
    w.get(u);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = u[j];
  } else {
    float u[8];
    unpack8(load8(p, n), u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = u[j];
  }
}

// 1 / sqrt(v), v > 0: the hardware's root takes numbers below 2^-126 for 0.
__device__ __forceinline__ float inv_root(float v) {
  const bool tiny = v < 1e-30f;
  return rsqrtf(tiny ? v * 0x1p96f : v) * (tiny ? 0x1p48f : 1.0f);
}

// What brings a row whose squares add to more than fp32 holds into the middle of
// its range: 512 squares of 2^128 2^-80 stay below 2^106, and what goes below the
// smallest number on the way is none of a row of 2^59 or more.  Its r is rounded to
// the subnormal step 2^-149 where the row's mean size is above 2^126: 2^-22 at most.
constexpr float kDown = 0x1p-80f;

// One row's place: offsets of its tensors, and its token's word of positions (or,
// without positions, its row of the table).
struct Place {
  int64_t x, dy, out, pos;
};
__device__ __forceinline__ Place place(const HeadRows& h, uint32_t r) {
  const uint32_t a = quotient(r, h.n0), i0 = r - a * h.n0.d, i2 = quotient(a, h.n1), i1 = a - i2 * h.n1.d;
  auto at = [&](const int64_t(&s)[3]) { return i0 * s[0] + i1 * s[1] + i2 * s[2]; };
  return {at(h.s_x), at(h.s_dy), at(h.s_out), at(h.s_pos)};
}

// The angles of a lane's 8 pairs, in runs that lie apart like its pieces.
template <typename T, bool INTER> struct Angles {
  static constexpr int LEN = INTER ? Piece<T>::N / 2 : Piece<T>::N, RUNS = 8 / LEN;
  float c[8], s[8];
  int n[RUNS];
};
template <int RAG, typename T, bool INTER>
__device__ __forceinline__ void load_angles(const HeadArgs& a, int64_t pos, const LanePart<T>& p, bool live,
                                            Angles<T, INTER>& g) {
  constexpr int LEN = Angles<T, INTER>::LEN;
  const int half = a.rot / 2;
  const bool turned = live && p.turned && half > 0;
  const int64_t row = turned && a.positions ? a.positions[pos] : pos;
  const bool in = turned && uint64_t(row) < uint64_t(a.table_rows);
#pragma unroll
  for (int i = 0; i < Angles<T, INTER>::RUNS; ++i) {
    const int at = INTER ? p.c[i] / 2 : p.c[i];
    int n = in ? some(half - at, LEN) : 0;
    if constexpr (!ragged_angles(RAG, INTER)) n = n > 0 ? LEN : 0;
    g.n[i] = n;
    if constexpr (ragged_angles(RAG, INTER) && LEN == 8) {
      const int left = n > 0 ? half - at : 0;
      Raw8<float> c = load_row8(a.cos + row * half, unsigned(at), left, half);
      Raw8<float> s = load_row8(a.sin + row * half, unsigned(at), left, half);
      settle8(c, left, half);
      settle8(s, left, half);
      float u[8];
      unpack8(c, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) g.c[j] = u[j];
      unpack8(s, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) g.s[j] = u[j];
    } else {
      load_run<LEN>(a.cos + row * half + at, n, g.c + LEN * i);
      load_run<LEN>(a.sin + row * half + at, n, g.s + LEN * i);
    }
  }
}

// Turns a lane's elements by its angles, or back.
template <int RAG, bool BACK, typename T, bool INTER>
__device__ __forceinline__ void turn(const Angles<T, INTER>& g, float (&v)[16]) {
  constexpr int LEN = Angles<T, INTER>::LEN;
#pragma unroll
  for (int i = 0; i < Angles<T, INTER>::RUNS; ++i) {
    if (g.n[i] <= 0) continue;
#pragma unroll
    for (int j = 0; j < LEN; ++j) {
      const int k = LEN * i + j;
      if (ragged_angles(RAG, INTER) && j >= g.n[i]) continue;
      float &a = v[INTER ? 2 * k : k], &b = v[INTER ? 2 * k + 1 : k + 8];
      const float s = BACK ? -g.s[k] : g.s[k];
      const float x = fmaf(a, g.c[k], -(b * s)), y = fmaf(b, g.c[k], a * s);
      a = x;
      b = y;
    }
  }
}

// A group of rows a workgroup, queries' workgroups before the keys'.  Bound by
// memory: 4 x 4096 tokens of 32 + 8 heads of 128 bf16, slices of a projection's
// output to heads before tokens, 66 us, 5.1 TB/s of the bytes that it cannot do
// without; 289 instructions a wave, 58 % of the cycles.  Two and four groups a
// workgroup 68.8 and 69.1 (the graph of that call 67.9), rows in the order of the
// output instead of the input 79, tiles of 4 heads by 8 tokens 73.
template <typename T, int LANES, bool INTER, int RAG>
__global__ __launch_bounds__(WG) void heads_fwd_kernel(HeadArgs a) {
  constexpr int ROWS = WG / LANES;
  const bool keys = int(blockIdx.x) >= a.q.wgs;
  const HeadRows& h = keys ? a.k : a.q;
  const uint32_t wg = keys ? blockIdx.x - a.q.wgs : blockIdx.x;
  const LanePart<T> p = lane_part<RAG, T, INTER>(threadIdx.x % LANES, a.dim, a.rot);
  const float inv = 1.0f / float(a.dim);
  float gv[16];
  load_gamma<RAG>(h.gamma, a.wbf16, p, a.dim, gv);
  for (uint64_t row = uint64_t(wg) * ROWS + threadIdx.x / LANES; row < h.rows; row += uint64_t(h.wgs) * ROWS) {
    const Place at = place(h, uint32_t(row));
    Held<T> held;
    Angles<T, INTER> ang;
    load_held<RAG>((const T*)h.x + at.x, p, true, a.dim, held);
    load_angles<RAG>(a, at.pos, p, true, ang);
    float v[16];
    unpack_held<RAG>(held, p, true, a.dim, v);
    float w[16], q = 0.0f;
    counted<RAG>(p, v, w);
#pragma unroll
    for (int j = 0; j < 16; ++j) q = fmaf(w[j], w[j], q);
    q = lane_sum<LANES>(q);
    float r = inv_root(fmaf(q, inv, a.eps));
    if (q == INFINITY) {  // squares beyond fp32: of the row scaled down
      q = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float d = v[j] * kDown;
        q = skipped<RAG>(p, j) ? q : fmaf(d, d, q);
      }
      r = inv_root(fmaf(lane_sum<LANES>(q), inv, a.eps * kDown * kDown)) * kDown;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = v[j] * r * gv[j];
    turn<RAG, false>(ang, v);
    store_held<RAG>((T*)h.out + at.out, p, true, v, a.stream_out);
  }
}

// At most kHeadMaxParts workgroups take every h.wgs-th group of rows and keep the
// sums of dgamma in registers.  r is formed again from x, which is read anyway.
// Bound by memory for many rows: 2 x 8192 tokens of 64 + 8 heads of 128 bf16 166 us,
// 5.5 TB/s, and 5 for the join; 49 % of the cycles are instructions.  768
// workgroups 173 (of a graph's 172), 512 185, 2048 199; with the next rows' loads
// in flight over the sums 173 with 768 workgroups, 205 with 1024 (three waves a
// SIMD instead of four).  64 tokens: 7.2 us, launches and latency.
// Four waves a SIMD are asked for: left to itself the compiler takes the registers of
// three for fp32 interleaved pairs of odd heads (2 x 4096 tokens of 12 + 4 heads of 33
// 26.8 us, 22.3 so); where pieces overlap it would spill.
template <typename T, int LANES, bool INTER, int RAG>
__global__ __launch_bounds__(WG, RAG == kOverlap ? 1 : 4) void heads_bwd_kernel(HeadArgs a) {
  constexpr int ROWS = WG / LANES, WAVES = WG / 64;
  __shared__ float sums[WAVES][16 * LANES];
  const bool keys = int(blockIdx.x) >= a.q.wgs;
  const HeadRows& h = keys ? a.k : a.q;
  const uint32_t wg = keys ? blockIdx.x - a.q.wgs : blockIdx.x;
  const LanePart<T> p = lane_part<RAG, T, INTER>(threadIdx.x % LANES, a.dim, a.rot);
  const float inv = 1.0f / float(a.dim);
  float gv[16], acc[16];
  load_gamma<RAG>(h.gamma, a.wbf16, p, a.dim, gv);
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = 0.0f;
  const uint64_t step = uint64_t(h.wgs) * ROWS;
  for (uint64_t row0 = uint64_t(wg) * ROWS; row0 < h.rows; row0 += step) {
    const uint64_t row = row0 + threadIdx.x / LANES;
    const bool live = row < h.rows;
    const Place at = place(h, live ? uint32_t(row) : h.rows - 1);
    Held<T> hx, hy;
    Angles<T, INTER> ang;
    load_held<RAG>((const T*)h.x + at.x, p, live, a.dim, hx);
    load_held<RAG>((const T*)h.dy + at.dy, p, live, a.dim, hy);
    load_angles<RAG>(a, at.pos, p, live, ang);
    float x[16], g[16];
    unpack_held<RAG>(hx, p, live, a.dim, x);
    unpack_held<RAG>(hy, p, live, a.dim, g);
    turn<RAG, true>(ang, g);
    float w[16], q = 0.0f, dot = 0.0f;
    counted<RAG>(p, x, w);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      q = fmaf(w[j], w[j], q);
      dot = fmaf(g[j] * gv[j], w[j], dot);
    }
    q = lane_sum<LANES>(q);
    dot = lane_sum<LANES>(dot);
    // The sums again: squares beyond fp32, of the row scaled down; or an infinite
    // gradient in an element that another lane counts, which has met the 0 above
    // (taking it out in every row takes the registers of a fourth wave: 2 x 4096 tokens
    // of 24 + 8 heads of 90 bf16 44.4 us, 37.1 so).
    float eps = a.eps, back = 1.0f;
    if (q == INFINITY || (RAG == kOverlap && dot != dot)) {
      if (q == INFINITY) {
        eps = eps * kDown * kDown;
        back = kDown;
      }
      q = dot = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        x[j] *= back;
        q = skipped<RAG>(p, j) ? q : fmaf(x[j], x[j], q);
        dot = skipped<RAG>(p, j) ? dot : fmaf(g[j] * gv[j], x[j], dot);
      }
      q = lane_sum<LANES>(q);
      dot = lane_sum<LANES>(dot);
    }
    const float r = inv_root(fmaf(q, inv, eps)), c = dot * r * inv, rx = r * back;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float xh = x[j] * r;
      acc[j] = fmaf(g[j], xh, acc[j]);
      x[j] = rx * fmaf(-xh, c, g[j] * gv[j]);
    }
    store_held<RAG>((T*)h.out + at.out, p, live, x, a.stream_out);
  }
  if (!h.dgamma) return;
  // the rows of a wave across its lanes, the waves in order
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = across_groups<LANES>(acc[j]);
  if ((threadIdx.x & 63) < LANES) {
    constexpr int E = LanePart<T>::E;
#pragma unroll
    for (int i = 0; i < LanePart<T>::P; ++i)
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (j >= p.skip[i] && j < p.n[i]) sums[threadIdx.x / 64][p.c[i] + j] = acc[E * i + j];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.dim; c += WG) {
    float s = sums[0][c];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += sums[w][c];
    if (h.part) h.part[int64_t(wg) * a.dim + c] = s;
    else if (a.wbf16) Elem<uint16_t>::store((uint16_t*)h.dgamma + c, s);
    else Elem<float>::store((float*)h.dgamma + c, s);
  }
}

// Joins the workgroups' sums (5 us for 1024 of 128 columns): 16 columns a
// workgroup, 64 slices of the at most 1024 parts, whose at most 16 loads are in
// flight at once; the slices of a wave are joined across its lanes, the waves in
// order.  blockIdx.y 0 for queries, 1 for keys.
constexpr int kCols = 16, kSlices = 64;
__global__ __launch_bounds__(kCols* kSlices) void heads_gain_kernel(HeadArgs a) {
  constexpr int EACH = (kHeadMaxParts + kSlices - 1) / kSlices, WAVES = kCols * kSlices / 64;
  __shared__ float sums[WAVES][kCols];
  const HeadRows& h = blockIdx.y ? a.k : a.q;
  if (!h.dgamma || !h.part) return;
  const int lane = threadIdx.x % kCols, slice = threadIdx.x / kCols, c = int(blockIdx.x) * kCols + lane;
  float v[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int p = slice + kSlices * i;
    v[i] = c < a.dim && p < h.wgs ? h.part[int64_t(p) * a.dim + c] : 0.0f;
  }
  float s = v[0];
#pragma unroll
  for (int i = 1; i < EACH; ++i) s += v[i];
  s = across_groups<kCols>(s);
  if ((threadIdx.x & 63) < kCols) sums[threadIdx.x / 64][lane] = s;
  __syncthreads();
  if (threadIdx.x < kCols && c < a.dim) {
#pragma unroll
    for (int i = 1; i < WAVES; ++i) s += sums[i][lane];
    if (a.wbf16) Elem<uint16_t>::store((uint16_t*)h.dgamma + c, s);
    else Elem<float>::store((float*)h.dgamma + c, s);
  }
}

// Sets the gradients of a call without rows to 0.
__global__ __launch_bounds__(WG) void heads_zero_kernel(HeadArgs a) {
  for (int c = threadIdx.x; c < a.dim; c += WG) {
    for (void* d : {a.q.dgamma, a.k.dgamma}) {
      if (!d) continue;
      if (a.wbf16) ((uint16_t*)d)[c] = 0;
      else ((float*)d)[c] = 0.0f;
    }
  }
}

template <typename F> hipError_t by_kind(const HeadArgs& a, bool bf16, bool inter, F f) {
  auto lanes = [&](auto t, auto in, auto rag) {
    constexpr int most = head_most_lanes(decltype(in)::value, decltype(rag)::value == kWhole, sizeof(t));
    switch (head_lanes(a.dim, a.rot, inter)) {
      case 4: f(t, in, rag, std::integral_constant<int, 4>{}); break;
      case 8: f(t, in, rag, std::integral_constant<int, 8>{}); break;
      case 16: f(t, in, rag, std::integral_constant<int, 16>{}); break;
      case 32: f(t, in, rag, std::integral_constant<int, 32>{}); break;
      default: if constexpr (most > 32) f(t, in, rag, std::integral_constant<int, 64>{});
    }
  };
  typedef std::integral_constant<int, kWhole> Whole;
  typedef std::integral_constant<int, kRaggedAngles> RaggedAngles;
  typedef std::integral_constant<int, kOverlap> Overlap;
  typedef std::integral_constant<int, kRagged> AllRagged;
  const int half = a.rot / 2, rest = a.dim - a.rot;
  auto kind = [&](auto t) {
    constexpr int E = Piece<decltype(t)>::N;
    if (inter) {
      if (a.dim % E == 0 && half % (E / 2) == 0) lanes(t, std::true_type{}, Whole{});
      else if (a.dim % E == 0) lanes(t, std::true_type{}, RaggedAngles{});
      else if (a.dim >= E && a.dim % 2 == 0) lanes(t, std::true_type{}, Overlap{});
      else lanes(t, std::true_type{}, AllRagged{});
    } else {
      if (half % E == 0 && rest % E == 0) lanes(t, std::false_type{}, Whole{});
      else if ((half == 0 || half >= E) && (rest == 0 || rest >= E)) lanes(t, std::false_type{}, Overlap{});
      else lanes(t, std::false_type{}, AllRagged{});
    }
  };
  bf16 ? kind(uint16_t{}) : kind(float{});
  return hipGetLastError();
}

// Whether the outputs are written past the caches: large ones (kStreamOut) whose
// runs of pieces are whole lines of 128 bytes, 8 lanes.  4 x 4096 tokens of 24 + 8
// heads of 128 bf16 forward 53.9 us, 57.1 without, backward 83.4 and 87.0; but heads
// of 112, of 7 lanes, 73.9 and 60.3, 89.2 and 81.0, and of 64 fp32 60.8 and 58.4.
bool streams(const HeadArgs& a, int64_t size, bool inter) {
  const int first = inter ? 0 : (a.rot / 2 + 7) / 8, others = ((inter ? a.dim : a.dim - a.rot) + 15) / 16;
  return first % 8 == 0 && others % 8 == 0 && (int64_t(a.q.rows) + a.k.rows) * a.dim * size > kStreamOut;
}

}  // namespace

hipError_t run_heads_fwd(const HeadArgs& args, bool bf16, bool interleaved, hipStream_t st) {
  return by_kind(args, bf16, interleaved, [&](auto t, auto inter, auto rag, auto lanes) {
    constexpr int L = decltype(lanes)::value, ROWS = WG / L;
    HeadArgs a = args;
    auto need = [](uint32_t rows) { return int(std::min<int64_t>((int64_t(rows) + ROWS - 1) / ROWS, kOpsMaxGrid)); };
    a.q.wgs = need(a.q.rows);
    a.k.wgs = need(a.k.rows);
    a.stream_out = streams(a, sizeof(t), interleaved);
    hipLaunchKernelGGL((heads_fwd_kernel<decltype(t), L, decltype(inter)::value, decltype(rag)::value>),
                       dim3(unsigned(a.q.wgs + a.k.wgs)), dim3(WG), 0, st, a);
  });
}

hipError_t run_heads_bwd(const HeadArgs& args, bool bf16, bool interleaved, hipStream_t st) {
  HeadArgs a = args;
  a.stream_out = streams(a, bf16 ? 2 : 4, interleaved);
  if (a.q.rows + a.k.rows == 0) {
    hipLaunchKernelGGL(heads_zero_kernel, dim3(1), dim3(WG), 0, st, a);
    return hipGetLastError();
  }
  const hipError_t e = by_kind(a, bf16, interleaved, [&](auto t, auto inter, auto rag, auto lanes) {
    constexpr int L = decltype(lanes)::value;
    hipLaunchKernelGGL((heads_bwd_kernel<decltype(t), L, decltype(inter)::value, decltype(rag)::value>),
                       dim3(unsigned(a.q.wgs + a.k.wgs)), dim3(WG), 0, st, a);
  });
  if (e != hipSuccess || !((a.q.dgamma && a.q.part) || (a.k.dgamma && a.k.part))) return e;
  hipLaunchKernelGGL(heads_gain_kernel, dim3(unsigned((a.dim + kCols - 1) / kCols), 2), dim3(kCols * kSlices), 0, st, a);
  return hipGetLastError();
}

}  // namespace muon
