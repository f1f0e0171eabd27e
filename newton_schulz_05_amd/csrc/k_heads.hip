// Norm of every query and key head with the position rotation, forward and
// backward:
//
//   forward   r = 1 / sqrt(mean(x^2) + eps), y = x r gamma, and in the first
//             rot elements every pair (a, b) turned by the token's angle,
//             (a c - b s, b c + a s)
//   backward  g = dy turned back, dgamma = sum over rows of g x r,
//             dx = r (g gamma - x r mean(g gamma x r))
//
// A head's row is read once and held by 4 to 64 lanes with two vectors of 8
// elements each.  Pairs that lie rot / 2 apart are one lane's two vectors, so
// turning needs no exchange between lanes.  Sums are fp32; each output is rounded
// once.
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

// What a lane holds of every row: n0 elements at column c0 and n1 at c1, of
// which the pairs up to nc are turned by the angles 8 t and on.
struct LanePart {
  int c0, c1, n0, n1, nc;
};
template <bool INTER> __device__ __forceinline__ LanePart lane_part(int t, int dim, int rot) {
  auto some = [](int n) { return n < 0 ? 0 : n > 8 ? 8 : n; };
  LanePart p;
  const int half = rot / 2, first = INTER ? 0 : (half + 7) / 8;
  if (INTER || t >= first) {
    p.c0 = (INTER ? 0 : rot) + 16 * (t - first);
    p.c1 = p.c0 + 8;
    p.n0 = some(dim - p.c0);
    p.n1 = some(dim - p.c1);
    p.nc = INTER ? some(half - 8 * t) : 0;
  } else {
    p.c0 = 8 * t;
    p.c1 = half + 8 * t;
    p.n0 = p.n1 = p.nc = some(half - 8 * t);
  }
  return p;
}

// n elements at col of a row of dim; with RAG the last ones behind n hold
// anything until settled, without it n is 0 or 8.
template <bool RAG, typename T>
__device__ __forceinline__ Raw8<T> load_part(const T* row, int col, int n, int dim) {
  if constexpr (RAG) return load_row8(row, unsigned(col), n > 0 ? dim - col : 0, dim);
  else return load8(row + col, n > 0 ? 8 : 0);
}
template <bool RAG, typename T> __device__ __forceinline__ void store_part(T* p, int n, const Raw8<T>& r) {
  store8(p, RAG ? n : (n > 0 ? 8 : 0), r);
}
template <bool RAG, typename T>
__device__ __forceinline__ void unpack_part(Raw8<T> r, int col, int n, int dim, float (&v)[8]) {
  if constexpr (RAG) settle8(r, n > 0 ? dim - col : 0, dim);
  unpack8(r, v);
  if constexpr (RAG) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? v[j] : 0.0f;
  }
}

// gamma, in fp32 whatever it is stored in; 1 if null.
__device__ __forceinline__ void load_gamma(const void* gamma, bool bf16, int col, int n, float (&v)[8]) {
  if (!gamma) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 1.0f;
  } else if (bf16) {
    unpack8(load8((const uint16_t*)gamma + col, n), v);
  } else {
    unpack8(load8((const float*)gamma + col, n), v);
  }
}

// One row's place: offsets of its tensors, and the table's row of its angles
// (-1: not turned).
struct Place {
  int64_t x, dy, out, pos;
};
__device__ __forceinline__ Place place(const HeadRows& h, uint32_t r) {
  const uint32_t a = quotient(r, h.n0), i0 = r - a * h.n0.d, i2 = quotient(a, h.n1), i1 = a - i2 * h.n1.d;
  auto at = [&](const int64_t(&s)[3]) { return i0 * s[0] + i1 * s[1] + i2 * s[2]; };
  return {at(h.s_x), at(h.s_dy), at(h.s_out), at(h.s_pos)};
}

// The angles of a row for one lane.
struct Angles {
  Raw8<float> c, s;
  int n;
};
template <bool RAG>
__device__ __forceinline__ Angles load_angles(const HeadArgs& a, int64_t pos, int t, int n) {
  Angles r;
  const int half = a.rot / 2;
  const int64_t row = n > 0 && a.positions ? a.positions[pos] : pos;
  r.n = uint64_t(row) < uint64_t(a.table_rows) ? n : 0;
  r.c = load_part<RAG>(a.cos + row * half, 8 * t, r.n, half);
  r.s = load_part<RAG>(a.sin + row * half, 8 * t, r.n, half);
  if constexpr (RAG) {
    settle8(r.c, r.n > 0 ? half - 8 * t : 0, half);
    settle8(r.s, r.n > 0 ? half - 8 * t : 0, half);
  }
  return r;
}

// Turns a lane's elements by its angles, or back.
template <bool INTER, bool RAG, bool BACK>
__device__ __forceinline__ void turn(const Angles& g, float (&u)[8], float (&v)[8]) {
  float c[8], s[8];
  unpack8(g.c, c);
  unpack8(g.s, s);
  auto pair = [&](int j, float& a, float& b) {
    const float w = BACK ? -s[j] : s[j];
    const float x = fmaf(a, c[j], -(b * w)), y = fmaf(b, c[j], a * w);
    a = x;
    b = y;
  };
  auto one = [&](int j) {
    if constexpr (!INTER) pair(j, u[j], v[j]);
    else if (j < 4) pair(j, u[2 * j], u[2 * j + 1]);
    else pair(j, v[2 * (j - 4)], v[2 * (j - 4) + 1]);
  };
  if (g.n == 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) one(j);
  } else if (g.n > 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < g.n) one(j);
  }
}

template <typename T, int LANES, bool INTER, bool RAG>
__global__ __launch_bounds__(WG) void heads_fwd_kernel(HeadArgs a) {
  constexpr int ROWS = WG / LANES;
  const bool keys = int(blockIdx.x) >= a.q.wgs;
  const HeadRows& h = keys ? a.k : a.q;
  const uint32_t wg = keys ? blockIdx.x - a.q.wgs : blockIdx.x;
  const int t = threadIdx.x % LANES;
  const LanePart p = lane_part<INTER>(t, a.dim, a.rot);
  const float inv = 1.0f / float(a.dim);
  float ga[8], gb[8];
  load_gamma(h.gamma, a.wbf16, p.c0, p.n0, ga);
  load_gamma(h.gamma, a.wbf16, p.c1, p.n1, gb);
  for (uint64_t row = uint64_t(wg) * ROWS + threadIdx.x / LANES; row < h.rows; row += uint64_t(h.wgs) * ROWS) {
    const Place at = place(h, uint32_t(row));
    const T* x = (const T*)h.x + at.x;
    const Raw8<T> ra = load_part<RAG>(x, p.c0, p.n0, a.dim), rb = load_part<RAG>(x, p.c1, p.n1, a.dim);
    const Angles ang = load_angles<RAG>(a, at.pos, t, p.nc);
    float u[8], v[8];
    unpack_part<RAG>(ra, p.c0, p.n0, a.dim, u);
    unpack_part<RAG>(rb, p.c1, p.n1, a.dim, v);
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) q = fmaf(u[j], u[j], q);
#pragma unroll
    for (int j = 0; j < 8; ++j) q = fmaf(v[j], v[j], q);
    q = lane_sum<LANES>(q);
    const float r = rsqrtf(fmaf(q, inv, a.eps));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u[j] = u[j] * r * ga[j];
      v[j] = v[j] * r * gb[j];
    }
    turn<INTER, RAG, false>(ang, u, v);
    T* out = (T*)h.out + at.out;
    store_part<RAG>(out + p.c0, p.n0, pack8(u, (const T*)nullptr));
    store_part<RAG>(out + p.c1, p.n1, pack8(v, (const T*)nullptr));
  }
}

template <typename T, int LANES, bool INTER, bool RAG>
__global__ __launch_bounds__(WG) void heads_bwd_kernel(HeadArgs a) {
  constexpr int ROWS = WG / LANES, WAVES = WG / 64;
  __shared__ float sums[WAVES][16 * LANES];
  const bool keys = int(blockIdx.x) >= a.q.wgs;
  const HeadRows& h = keys ? a.k : a.q;
  const uint32_t wg = keys ? blockIdx.x - a.q.wgs : blockIdx.x;
  const int t = threadIdx.x % LANES;
  const LanePart p = lane_part<INTER>(t, a.dim, a.rot);
  const float inv = 1.0f / float(a.dim);
  float ga[8], gb[8], da[8], db[8];
  load_gamma(h.gamma, a.wbf16, p.c0, p.n0, ga);
  load_gamma(h.gamma, a.wbf16, p.c1, p.n1, gb);
#pragma unroll
  for (int j = 0; j < 8; ++j) da[j] = db[j] = 0.0f;
  const uint64_t step = uint64_t(h.wgs) * ROWS;
  for (uint64_t row0 = uint64_t(wg) * ROWS; row0 < h.rows; row0 += step) {
    const uint64_t row = row0 + threadIdx.x / LANES;
    const bool live = row < h.rows;
    const Place at = place(h, live ? uint32_t(row) : h.rows - 1);
    const int n0 = live ? p.n0 : 0, n1 = live ? p.n1 : 0;
    const T *x = (const T*)h.x + at.x, *dy = (const T*)h.dy + at.dy;
    const Raw8<T> xa = load_part<RAG>(x, p.c0, n0, a.dim), xb = load_part<RAG>(x, p.c1, n1, a.dim);
    const Raw8<T> ya = load_part<RAG>(dy, p.c0, n0, a.dim), yb = load_part<RAG>(dy, p.c1, n1, a.dim);
    const Angles ang = load_angles<RAG>(a, at.pos, t, live ? p.nc : 0);
    float u[8], v[8], g[8], f[8];
    unpack_part<RAG>(xa, p.c0, n0, a.dim, u);
    unpack_part<RAG>(xb, p.c1, n1, a.dim, v);
    unpack_part<RAG>(ya, p.c0, n0, a.dim, g);
    unpack_part<RAG>(yb, p.c1, n1, a.dim, f);
    turn<INTER, RAG, true>(ang, g, f);
    float q = 0.0f, dot = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      q = fmaf(u[j], u[j], q);
      dot = fmaf(g[j] * ga[j], u[j], dot);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      q = fmaf(v[j], v[j], q);
      dot = fmaf(f[j] * gb[j], v[j], dot);
    }
    q = lane_sum<LANES>(q);
    dot = lane_sum<LANES>(dot);
    const float r = rsqrtf(fmaf(q, inv, a.eps)), c = dot * r * inv;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float xu = u[j] * r, xv = v[j] * r;
      da[j] = fmaf(g[j], xu, da[j]);
      db[j] = fmaf(f[j], xv, db[j]);
      u[j] = r * fmaf(-xu, c, g[j] * ga[j]);
      v[j] = r * fmaf(-xv, c, f[j] * gb[j]);
    }
    T* out = (T*)h.out + at.out;
    store_part<RAG>(out + p.c0, n0, pack8(u, (const T*)nullptr));
    store_part<RAG>(out + p.c1, n1, pack8(v, (const T*)nullptr));
  }
  if (!h.dgamma) return;
  // the rows of a wave across its lanes, the waves in order
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    da[j] = across_groups<LANES>(da[j]);
    db[j] = across_groups<LANES>(db[j]);
  }
  if ((threadIdx.x & 63) < LANES) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < p.n0) sums[threadIdx.x / 64][p.c0 + j] = da[j];
      if (j < p.n1) sums[threadIdx.x / 64][p.c1 + j] = db[j];
    }
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

// Joins the workgroups' sums: 32 columns a workgroup, 32 slices of the parts,
// joined in order; blockIdx.y 0 for queries, 1 for keys.
constexpr int kCols = 32, kSlices = 32;
__global__ __launch_bounds__(kCols* kSlices) void heads_gain_kernel(HeadArgs a) {
  __shared__ float sums[kSlices][kCols];
  const HeadRows& h = blockIdx.y ? a.k : a.q;
  if (!h.dgamma || !h.part) return;
  const int lane = threadIdx.x % kCols, slice = threadIdx.x / kCols, c = int(blockIdx.x) * kCols + lane;
  float s = 0.0f;
#pragma unroll 8
  for (int p = slice; p < h.wgs; p += kSlices) s += c < a.dim ? h.part[int64_t(p) * a.dim + c] : 0.0f;
  sums[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < a.dim) {
#pragma unroll
    for (int i = 1; i < kSlices; ++i) s += sums[i][lane];
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
    switch (head_lanes(a.dim, a.rot, inter)) {
      case 4: f(t, in, rag, std::integral_constant<int, 4>{}); break;
      case 8: f(t, in, rag, std::integral_constant<int, 8>{}); break;
      case 16: f(t, in, rag, std::integral_constant<int, 16>{}); break;
      case 32: f(t, in, rag, std::integral_constant<int, 32>{}); break;
      default: f(t, in, rag, std::integral_constant<int, 64>{});
    }
  };
  // whole vectors only: the halves' and the rest's lengths are multiples of 8
  const bool rag = a.dim % 8 != 0 || (!inter && a.rot / 2 % 8 != 0) || (inter && a.rot % 16 != 0);
  auto kind = [&](auto t) {
    if (inter) rag ? lanes(t, std::true_type{}, std::true_type{}) : lanes(t, std::true_type{}, std::false_type{});
    else rag ? lanes(t, std::false_type{}, std::true_type{}) : lanes(t, std::false_type{}, std::false_type{});
  };
  bf16 ? kind(uint16_t{}) : kind(float{});
  return hipGetLastError();
}

}  // namespace

hipError_t run_heads_fwd(const HeadArgs& args, bool bf16, bool interleaved, hipStream_t st) {
  return by_kind(args, bf16, interleaved, [&](auto t, auto inter, auto rag, auto lanes) {
    constexpr int L = decltype(lanes)::value, ROWS = WG / L;
    HeadArgs a = args;
    auto need = [](uint32_t rows) { return int(std::min<int64_t>((int64_t(rows) + ROWS - 1) / ROWS, kOpsMaxGrid)); };
    a.q.wgs = need(a.q.rows);
    a.k.wgs = need(a.k.rows);
    hipLaunchKernelGGL((heads_fwd_kernel<decltype(t), L, decltype(inter)::value, decltype(rag)::value>),
                       dim3(unsigned(a.q.wgs + a.k.wgs)), dim3(WG), 0, st, a);
  });
}

hipError_t run_heads_bwd(const HeadArgs& a, bool bf16, bool interleaved, hipStream_t st) {
  if (a.q.rows + a.k.rows == 0) {
    hipLaunchKernelGGL(heads_zero_kernel, dim3(1), dim3(WG), 0, st, a);
    return hipGetLastError();
  }
  const hipError_t e = by_kind(a, bf16, interleaved, [&](auto t, auto inter, auto rag, auto lanes) {
    hipLaunchKernelGGL((heads_bwd_kernel<decltype(t), decltype(lanes)::value, decltype(inter)::value, decltype(rag)::value>),
                       dim3(unsigned(a.q.wgs + a.k.wgs)), dim3(WG), 0, st, a);
  });
  if (e != hipSuccess || !((a.q.dgamma && a.q.part) || (a.k.dgamma && a.k.part))) return e;
  hipLaunchKernelGGL(heads_gain_kernel, dim3(unsigned((a.dim + kCols - 1) / kCols), 2), dim3(kCols * kSlices), 0, st, a);
  return hipGetLastError();
}

}  // namespace muon
