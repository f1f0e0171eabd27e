// Layer norm, backward (see norm_dev.hpp).
#include "norm_dev.hpp"

namespace muon {

namespace {

// Two sums over the NT threads of a row with one barrier (see row_sum; `red`
// alternates from row to row).
template <int NT> __device__ __forceinline__ void row_sum2(float& a, float& b, float (*red)[2]) {
  if constexpr (NT <= 64) {
    a = lane_sum<NT>(a);
    b = lane_sum<NT>(b);
  } else {
    constexpr int NW = NT / 64;
    a = lane_sum<64>(a);
    b = lane_sum<64>(b);
    const int wave = threadIdx.x / 64, first = wave / NW * NW;
    if (threadIdx.x % 64 == 0) {
      red[wave][0] = a;
      red[wave][1] = b;
    }
    __syncthreads();
    a = red[first][0];
    b = red[first][1];
#pragma unroll
    for (int i = 1; i < NW; ++i) {
      a += red[first + i][0];
      b += red[first + i][1];
    }
  }
}

// One thread's vectors of a row.
template <typename T, int NV> struct RowPart {
  Raw8<T> x[NV], dy[NV], dh[NV];
  float mean, rstd;
};

template <typename T, int NT, int NV, bool FUSED, bool RAG>
__device__ __forceinline__ void fetch_row(const NormBwdArgs& a, int64_t row, int t, RowPart<T, NV>& r) {
  const bool live = row < a.rows;
  r.mean = live ? a.mean[row] : 0.0f;
  r.rstd = live ? a.rstd[row] : 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const unsigned col = 8 * (i * NT + opaque(t));
    const int n = live ? a.cols - int(col) : 0;
    r.x[i] = load_vec<RAG>((const T*)a.x + row * a.ld_x, col, n, a.cols);
    r.dy[i] = load_vec<RAG>((const T*)a.dy + row * a.ld_dy, col, n, a.cols);
    if constexpr (FUSED)
      if (a.dh) r.dh[i] = load_vec<RAG>((const T*)a.dh + row * a.ld_dh, col, n, a.cols);
  }
}

template <typename T, int NT, int NV, bool FUSED, bool RAG>
__device__ __forceinline__ void settle_row(const NormBwdArgs& a, bool live, int t, RowPart<T, NV>& r) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int n = live ? a.cols - 8 * (i * NT + opaque(t)) : 0;
    settle<RAG>(r.x[i], n, a.cols);
    settle<RAG>(r.dy[i], n, a.cols);
    if constexpr (FUSED)
      if (a.dh) settle<RAG>(r.dh[i], n, a.cols);
  }
}

// Hides a vector's bits from the optimiser: what was computed from them before
// a row's reduction is computed again after it, instead of being kept in
// registers over it (the unpacked row is twice the packed one in bf16).
__device__ __forceinline__ void hide(Raw8<uint16_t>& v) { asm volatile("" : "+v"(v.w)); }
__device__ __forceinline__ void hide(Raw8<float>& v) { asm volatile("" : "+v"(v.a), "+v"(v.b)); }

// Stores dx of one vector, and with FUSED dres.
template <typename T, typename W, bool FUSED, bool RAG>
__device__ __forceinline__ void emit_dx(const NormBwdArgs& a, int64_t row, unsigned col, int n, const Raw8<T>& xr,
                                        const Raw8<T>& dr, const Raw8<T>& hr, const float (&gv)[8], float mean,
                                        float rstd, float c1, float c2, uint64_t off) {
  float xv[8], dv[8];
  unpack8(xr, xv);
  unpack8(dr, dv);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float xh = (xv[j] - mean) * rstd, g = dv[j] * gv[j];
    dv[j] = rstd * fmaf(-xh, c2, g - c1);
  }
  if constexpr (FUSED) {
    if (a.dh) {
      unpack8(hr, xv);
#pragma unroll
      for (int j = 0; j < 8; ++j) dv[j] += xv[j];
    }
    store_vec<RAG>((T*)a.dres + row * a.ld_dres + col, n, pack8(dv, (const T*)nullptr));
    const u32x4 w = drop_draws(a.drop, off, uint32_t(row), col / 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) dv[j] = drop_keeps(w, j, a.drop.thresh) ? dv[j] * a.drop.scale : 0.0f;
  }
  store_vec<RAG>((T*)a.dx + row * a.ld_dx + col, n, pack8(dv, (const T*)nullptr));
}

// dgamma and dbeta of 64 columns over all rows, for few rows: 8 threads take the
// columns' vectors of a row, the others the further rows; a wave's rows are
// joined across its lanes, the waves in LDS.
template <typename T, typename W, int WG, bool RAG>
__device__ __forceinline__ void few_rows_sums(const NormBwdArgs& a, int strip, float (*sums)[2][64]) {
  const int vec = threadIdx.x & 7, wave = threadIdx.x >> 6;
  const unsigned col = strip * 64 + vec * 8;
  const int n = a.cols - int(col);
  float dg[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dg[j] = db[j] = 0.0f;
  for (int64_t row = threadIdx.x >> 3; row < a.rows; row += WG / 8) {
    float xv[8], dv[8];
    Raw8<T> xr = load_vec<RAG>((const T*)a.x + row * a.ld_x, col, n, a.cols);
    Raw8<T> dr = load_vec<RAG>((const T*)a.dy + row * a.ld_dy, col, n, a.cols);
    settle<RAG>(xr, n, a.cols);
    settle<RAG>(dr, n, a.cols);
    unpack8(xr, xv);
    unpack8(dr, dv);
    const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dg[j] = fmaf(dv[j], (xv[j] - mean) * rstd, dg[j]);
      db[j] += dv[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    dg[j] = across_groups<8>(dg[j]);
    db[j] = across_groups<8>(db[j]);
  }
  if ((threadIdx.x & 63) < 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sums[wave][0][vec * 8 + j] = dg[j];
      sums[wave][1][vec * 8 + j] = db[j];
    }
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    const int part = threadIdx.x >> 6, c = threadIdx.x & 63;
    float s = sums[0][part][c];
#pragma unroll
    for (int w = 1; w < WG / 64; ++w) s += sums[w][part][c];
    W* out = (W*)(part ? a.dbeta : a.dgamma);
    if (out && strip * 64 + c < a.cols) Elem<W>::store(out + strip * 64 + c, s);
  }
}

// Where the sums over rows of dgamma and dbeta are formed.
enum NormSums {
  kSumsHere,   // in registers beside dx, one partial sum a workgroup
  kSumsApart,  // by another kernel
  kSumsFew,    // by the launch's last workgroups, a strip of 64 columns each
};

// Workgroups of WG threads take every gridDim.x-th group of WG / NT rows.  With
// kSumsHere a workgroup's row groups are joined in LDS in a fixed order, and the
// workgroups' sums by norm_grad_kernel.
//
// Bound by memory: x and dy are read and dx written once.  For many rows one
// workgroup of 1024 threads on each of 256 units, one 16-byte vector a thread
// (16 sums to keep), with the next row's loads in flight over the reduction
// (AHEAD), measured best: 16384 x 8192 bf16 149.6 us, 157.0 without AHEAD; 16384 x
// 4096 79.1 and 81.0.  The fused pass has a third stream in flight and gains
// nothing from it (16384 x 4096 129.1 without, 127.7 with), nor do two vectors a
// thread (4000 x 16384 88.9 without, 89.7 with).  Rows above 20480 columns have no
// registers for the sums: see norm_cols_kernel.
template <typename T, typename W, int NT, int NV, int WG, bool FUSED, bool RAG, NormSums WHERE>
__global__ __launch_bounds__(WG) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int RPB = WG / NT, JOIN = NT < 64 ? WG / 64 : RPB;
  constexpr bool SUMS = WHERE == kSumsHere, AHEAD = SUMS && !FUSED && NV == 1;
  __shared__ float red[2][WG / 64][2];
  __shared__ float sums[SUMS && JOIN > 1 ? JOIN : 1][SUMS && JOIN > 1 ? 8 * NT * NV : 1];
  if constexpr (WHERE == kSumsFew) {
    __shared__ float strips[WG / 64][2][64];
    const int first = int((a.rows + RPB - 1) / RPB);
    if (int(blockIdx.x) >= first) {
      few_rows_sums<T, W, WG, RAG>(a, int(blockIdx.x) - first, strips);
      return;
    }
  }
  const int t = threadIdx.x % NT, sub = row_group<NT>();
  const int cols = a.cols;
  Raw8<W> gr[NV];
  float dg[NV][8], db[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const unsigned col = 8 * (i * NT + opaque(t));
    gr[i] = load_param<RAG, W>(a.gamma, col, cols);
    settle<RAG>(gr[i], cols - int(col), cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = db[i][j] = 0.0f;
  }
  const uint64_t off = FUSED ? drop_offset(a.drop) : 0;
  const float inv = 1.0f / float(cols);
  const int64_t step = int64_t(gridDim.x) * RPB;
  RowPart<T, NV> r;
  if constexpr (AHEAD) fetch_row<T, NT, NV, FUSED, RAG>(a, int64_t(blockIdx.x) * RPB + sub, t, r);
  int side = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + sub;
    const bool live = row < a.rows;
    RowPart<T, NV> next;
    if constexpr (AHEAD) fetch_row<T, NT, NV, FUSED, RAG>(a, row + step, t, next);
    else fetch_row<T, NT, NV, FUSED, RAG>(a, row, t, r);
    settle_row<T, NT, NV, FUSED, RAG>(a, live, t, r);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float xv[8], dv[8], gv[8];
      unpack8(r.x[i], xv);
      unpack8(r.dy[i], dv);
      unpack_param(gr[i], a.gamma, 1.0f, gv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // dy is 0 in the elements behind the row's end
        const float xh = (xv[j] - r.mean) * r.rstd, g = dv[j] * gv[j];
        s1 += g;
        s2 = fmaf(g, xh, s2);
        if constexpr (SUMS) {
          dg[i][j] = fmaf(dv[j], xh, dg[i][j]);
          db[i][j] += dv[j];
        }
      }
    }
    row_sum2<NT>(s1, s2, red[side]);
    side ^= 1;
    // mean * rstd overflows only for rows whose elements all equal the mean,
    // where xh is 0 and s2 with it; lanes without an element have added 0 * inf
    const float c1 = s1 * inv, c2 = fabsf(r.mean * r.rstd) == INFINITY ? 0.0f : s2 * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const unsigned col = 8 * (i * NT + opaque(t));
      if constexpr (NV > 1) {
        hide(r.x[i]);
        hide(r.dy[i]);
        hide(gr[i]);
      }
      float gv[8];
      unpack_param(gr[i], a.gamma, 1.0f, gv);
      emit_dx<T, W, FUSED, RAG>(a, row, col, live ? cols - int(col) : 0, r.x[i], r.dy[i], r.dh[i], gv, r.mean, r.rstd, c1,
                           c2, off);
    }
    if constexpr (AHEAD) r = next;
  }
  if constexpr (SUMS) {
    if (!a.dgamma && !a.dbeta) return;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      float(&acc)[NV][8] = part ? db : dg;
      float* to = a.part + (int64_t(blockIdx.x) * 2 + part) * cols;
      if constexpr (JOIN > 1) {
        // the row groups of a wave across its lanes, then the waves or groups in order
        if constexpr (NT < 64) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = across_groups<NT>(acc[i][j]);
        }
        __syncthreads();
        if (NT >= 64 || (threadIdx.x & 63) < NT) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sums[NT < 64 ? threadIdx.x / 64 : sub][8 * (i * NT + t) + j] = acc[i][j];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += WG) {
          float s = sums[0][c];
#pragma unroll
          for (int g = 1; g < JOIN; ++g) s += sums[g][c];
          to[c] = s;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = 8 * (i * NT + t);
          store8(to + c, cols - c, pack8(acc[i], (const float*)nullptr));
        }
      }
    }
  }
}

// The sums of rows wider than 20480 columns, in a pass of its own over x and
// dy: blockIdx.x takes 2048 columns, a vector a thread, and blockIdx.y every
// gridDim.y-th row.  With the sums in norm_bwd_kernel four vectors a thread
// spilled (2048 x 32768 bf16: 288 us; 147 so).
template <typename T, bool RAG>
__global__ __launch_bounds__(256) void norm_cols_kernel(NormBwdArgs a) {
  const unsigned col = 8 * (blockIdx.x * 256 + threadIdx.x);
  const int n = a.cols - int(col);
  float dg[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dg[j] = db[j] = 0.0f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    float xv[8], dv[8];
    Raw8<T> xr = load_vec<RAG>((const T*)a.x + row * a.ld_x, col, n, a.cols);
    Raw8<T> dr = load_vec<RAG>((const T*)a.dy + row * a.ld_dy, col, n, a.cols);
    settle<RAG>(xr, n, a.cols);
    settle<RAG>(dr, n, a.cols);
    unpack8(xr, xv);
    unpack8(dr, dv);
    const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dg[j] = fmaf(dv[j], (xv[j] - mean) * rstd, dg[j]);
      db[j] += dv[j];
    }
  }
  float* to = a.part + int64_t(blockIdx.y) * 2 * a.cols;
  store8(to + col, n, pack8(dg, (const float*)nullptr));
  store8(to + a.cols + col, n, pack8(db, (const float*)nullptr));
}

// Sums the workgroups' partial dgamma (blockIdx.y == 0) and dbeta over
// `parts` <= 256: 32 columns a workgroup, 32 slices of the parts, whose at
// most 8 loads are all in flight at once; the slices are joined in order.
constexpr int kGradCols = 32, kGradSlices = 32;
template <typename W>
__global__ __launch_bounds__(kGradCols* kGradSlices) void norm_grad_kernel(const float* part, int parts, int cols,
                                                                           W* dgamma, W* dbeta) {
  __shared__ float sums[kGradSlices][kGradCols];
  W* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const int lane = threadIdx.x % kGradCols, slice = threadIdx.x / kGradCols;
  const int c = int(blockIdx.x) * kGradCols + lane;
  float v[kNormMaxParts / kGradSlices];
#pragma unroll
  for (int i = 0; i < kNormMaxParts / kGradSlices; ++i) {
    const int p = slice + kGradSlices * i;
    v[i] = c < cols && p < parts ? part[(int64_t(p) * 2 + blockIdx.y) * cols + c] : 0.0f;
  }
  float s = v[0];
#pragma unroll
  for (int i = 1; i < kNormMaxParts / kGradSlices; ++i) s += v[i];
  sums[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < kGradSlices; ++i) s += sums[i][lane];
    Elem<W>::store(out + c, s);
  }
}

template <typename T, typename W, bool FUSED, bool RAG> struct BwdLaunch {
  template <int NT, int NV, int WG> static void bwd(const NormBwdArgs& a, hipStream_t st) {
    hipLaunchKernelGGL((norm_bwd_kernel<T, W, NT, NV, WG, FUSED, RAG, kSumsHere>), dim3(unsigned(a.parts)), dim3(WG), 0, st,
                       a);
  }
  template <int NT> static void bwd(const NormBwdArgs& a, int wg, hipStream_t st) {
    wg == 256 ? bwd<NT, 1, 256>(a, st) : bwd<NT, 1, 1024>(a, st);
  }
  template <int NT, int NV> static void bwd_apart(const NormBwdArgs& a, bool grads, hipStream_t st) {
    hipLaunchKernelGGL((norm_bwd_kernel<T, W, NT, NV, NT, FUSED, RAG, kSumsApart>),
                       dim3(unsigned(std::min(a.rows, kOpsMaxGrid))), dim3(NT), 0, st, a);
    if (grads)
      hipLaunchKernelGGL((norm_cols_kernel<T, RAG>), dim3(unsigned((a.cols + 2047) / 2048), unsigned(a.parts)), dim3(256), 0,
                         st, a);
  }
  template <int NT, int NV> static void bwd_few(const NormBwdArgs& a, hipStream_t st) {
    constexpr int WG = NT < 256 ? 256 : NT;
    const int64_t groups = (a.rows + WG / NT - 1) / (WG / NT), strips = (a.dgamma || a.dbeta) ? (a.cols + 63) / 64 : 0;
    if (groups + strips > 0)
      hipLaunchKernelGGL((norm_bwd_kernel<T, W, NT, NV, WG, FUSED, RAG, kSumsFew>), dim3(unsigned(groups + strips)), dim3(WG),
                         0, st, a);
  }
  static hipError_t bwd(const NormBwdArgs& a, hipStream_t st) {
    const NormBwdSplit sp = norm_bwd_split(a.rows, a.cols);
    const bool grads = a.dgamma || a.dbeta;
    if (sp.parts == 0) {
      switch (sp.row_threads) {
        case 8: bwd_few<8, 1>(a, st); break;
        case 16: bwd_few<16, 1>(a, st); break;
        case 32: bwd_few<32, 1>(a, st); break;
        case 64: bwd_few<64, 1>(a, st); break;
        case 128: bwd_few<128, 1>(a, st); break;
        case 256: bwd_few<256, 1>(a, st); break;
        case 512: bwd_few<512, 1>(a, st); break;
        default:
          a.cols <= 8192 ? bwd_few<1024, 1>(a, st) : a.cols <= 16384 ? bwd_few<1024, 2>(a, st) : bwd_few<1024, 4>(a, st);
      }
      return hipGetLastError();
    }
    const int vecs = (a.cols + 7) / 8;
    switch (sp.row_threads) {
      case 8: bwd<8>(a, sp.threads, st); break;
      case 16: bwd<16>(a, sp.threads, st); break;
      case 32: bwd<32>(a, sp.threads, st); break;
      case 64: bwd<64>(a, sp.threads, st); break;
      case 128: bwd<128>(a, sp.threads, st); break;
      case 256: bwd<256, 1, 1024>(a, st); break;
      case 512: bwd<512, 1, 1024>(a, st); break;
      default:
        if (vecs <= 1024) bwd<1024, 1, 1024>(a, st);
        else if (vecs <= 1536) bwd<512, 3, 512>(a, st);
        else if (vecs <= 2048) bwd<1024, 2, 1024>(a, st);
        else if (vecs <= 2560) bwd<512, 5, 512>(a, st);
        else if (a.cols <= 24576) bwd_apart<1024, 3>(a, grads, st);
        else bwd_apart<1024, 4>(a, grads, st);
    }
    if (grads)
      hipLaunchKernelGGL((norm_grad_kernel<W>), dim3(unsigned((a.cols + kGradCols - 1) / kGradCols), 2),
                         dim3(kGradCols * kGradSlices), 0, st, a.part, a.parts, a.cols, (W*)a.dgamma, (W*)a.dbeta);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t run_norm_bwd(const NormBwdArgs& a, bool bf16, bool wbf16, bool fused, hipStream_t st) {
  return norm_by_types<BwdLaunch>(a.cols, bf16, wbf16, fused, [&](auto l) { return l.bwd(a, st); });
}

}  // namespace muon
