// Layer norm over the rows of [rows, cols], forward and backward, alone or
// fused with the residual add and dropout before it.
//
//   forward   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps),
//             y = (x - mu) r gamma + beta
//   backward  xh = (x - mu) r, g = dy gamma,
//             dx = r (g - mean(g) - xh mean(g xh)),
//             dgamma = sum over rows of dy xh, dbeta = sum over rows of dy
//   fused     h = residual + dropout(x), y = norm(h);
//             dh = norm backward + the gradient that reaches h directly,
//             dresidual = dh, dx = dropout of dh with the same mask
//
// A row is read once and held in registers by 16 to 1024 threads, so the mean
// comes before the squared deviations are formed (no cancellation) without a
// second pass over memory.  All sums are fp32; each output is rounded once.
#include "ops_dev.hpp"

// Products and sums are joined only where fmaf says so, so that every variant
// of a kernel (fused or not, any row split) rounds alike.
#pragma clang fp contract(off)

namespace muon {

namespace {

// Sum over the NT threads of a row; `red` holds one word per wave and row.
// The caller alternates two `red` buffers, so that one barrier per sum is
// enough.
template <int NT> __device__ __forceinline__ float row_sum(float v, float* red) {
  if constexpr (NT <= 64) {
    return lane_sum<NT>(v);
  } else {
    constexpr int NW = NT / 64;
    v = lane_sum<64>(v);
    const int wave = threadIdx.x / 64, first = wave / NW * NW;
    if (threadIdx.x % 64 == 0) red[wave] = v;
    __syncthreads();
    float s = red[first];
#pragma unroll
    for (int i = 1; i < NW; ++i) s += red[first + i];
    return s;
  }
}

template <typename T> __device__ __forceinline__ void load_param(const void* p, int col, int n, float dflt,
                                                                 float (&v)[8]) {
  if (p) {
    unpack8(load8((const T*)p + col, n), v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = dflt;
  }
}

template <typename T, typename W, int NT, int NV, int WG, bool FUSED>
__global__ __launch_bounds__(WG) void norm_fwd_kernel(NormFwdArgs a) {
  constexpr int RPB = WG / NT;
  __shared__ float red[2][WG / 64];
  const int t = threadIdx.x % NT, sub = threadIdx.x / NT;
  const int cols = a.cols;
  float gam[NV][8], bet[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = 8 * (i * NT + t);
    load_param<W>(a.gamma, col, cols - col, 1.0f, gam[i]);
    load_param<W>(a.beta, col, cols - col, 0.0f, bet[i]);
  }
  const uint64_t off = FUSED ? drop_offset(a.drop) : 0;
  for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < a.rows; row0 += int64_t(gridDim.x) * RPB) {
    const int64_t row = row0 + sub;
    const bool live = row < a.rows;
    float v[NV][8];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = 8 * (i * NT + t), n = live ? cols - col : 0;
      unpack8(load8((const T*)a.x + row * a.ld_x + col, n), v[i]);
      if constexpr (FUSED) {
        float rv[8];
        unpack8(load8((const T*)a.res + row * a.ld_res + col, n), rv);
        const u32x4 w = drop_draws(a.drop, off, uint32_t(row), uint32_t(col / 8));
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i][j] = drop_keeps(w, j, a.drop.thresh) ? fmaf(v[i][j], a.drop.scale, rv[j]) : rv[j];
        // the norm is that of h as it is stored, so that the backward pass,
        // which reads h, sees the same values
        const Raw8<T> hr = pack8(v[i], (const T*)nullptr);
        store8((T*)a.h + row * a.ld_h + col, n, hr);
        unpack8(hr, v[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s += j < n ? v[i][j] : 0.0f;
    }
    const float mean = row_sum<NT>(s, red[0]) / float(cols);
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int n = cols - 8 * (i * NT + t);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] -= mean;
        q = j < n ? fmaf(v[i][j], v[i][j], q) : q;
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<NT>(q, red[1]) / float(cols) + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = 8 * (i * NT + t), n = live ? cols - col : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * rstd, gam[i][j], bet[i][j]);
      store8((T*)a.y + row * a.ld_y + col, n, pack8(v[i], (const T*)nullptr));
    }
    if (live && t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// One workgroup takes every gridDim.x-th group of WG / NT rows and keeps the
// sums of its columns' dgamma and dbeta in registers; its row groups are
// joined in LDS in a fixed order, and the workgroups' sums by
// norm_grad_kernel.  A lone workgroup writes the gradients itself.
template <typename T, typename W, int NT, int NV, int WG, bool FUSED>
__global__ __launch_bounds__(WG) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int RPB = WG / NT;
  __shared__ float red[2][WG / 64];
  __shared__ float sums[RPB > 1 ? RPB : 1][RPB > 1 ? 8 * NT * NV : 1];
  const int t = threadIdx.x % NT, sub = threadIdx.x / NT;
  const int cols = a.cols;
  float gam[NV][8], dg[NV][8], db[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = 8 * (i * NT + t);
    load_param<W>(a.gamma, col, cols - col, 1.0f, gam[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = db[i][j] = 0.0f;
  }
  const uint64_t off = FUSED ? drop_offset(a.drop) : 0;
  const float inv = 1.0f / float(cols);
  for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < a.rows; row0 += int64_t(gridDim.x) * RPB) {
    const int64_t row = row0 + sub;
    const bool live = row < a.rows;
    const float mean = live ? a.mean[row] : 0.0f, rstd = live ? a.rstd[row] : 0.0f;
    Raw8<T> xr[NV], dr[NV];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = 8 * (i * NT + t), n = live ? cols - col : 0;
      xr[i] = load8((const T*)a.x + row * a.ld_x + col, n);
      dr[i] = load8((const T*)a.dy + row * a.ld_dy + col, n);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float xv[8], dv[8];
      unpack8(xr[i], xv);
      unpack8(dr[i], dv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // dy is 0 in the elements behind the row's end
        const float xh = (xv[j] - mean) * rstd, g = dv[j] * gam[i][j];
        s1 += g;
        s2 = fmaf(g, xh, s2);
        dg[i][j] = fmaf(dv[j], xh, dg[i][j]);
        db[i][j] += dv[j];
      }
    }
    const float c1 = row_sum<NT>(s1, red[0]) * inv, c2 = row_sum<NT>(s2, red[1]) * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = 8 * (i * NT + t), n = live ? cols - col : 0;
      float xv[8], dv[8];
      unpack8(xr[i], xv);
      unpack8(dr[i], dv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = (xv[j] - mean) * rstd, g = dv[j] * gam[i][j];
        dv[j] = rstd * fmaf(-xh, c2, g - c1);
      }
      if constexpr (FUSED) {
        if (a.dh) {
          unpack8(load8((const T*)a.dh + row * a.ld_dh + col, n), xv);
#pragma unroll
          for (int j = 0; j < 8; ++j) dv[j] += xv[j];
        }
        store8((T*)a.dres + row * a.ld_dres + col, n, pack8(dv, (const T*)nullptr));
        const u32x4 w = drop_draws(a.drop, off, uint32_t(row), uint32_t(col / 8));
#pragma unroll
        for (int j = 0; j < 8; ++j) dv[j] = drop_keeps(w, j, a.drop.thresh) ? dv[j] * a.drop.scale : 0.0f;
      }
      store8((T*)a.dx + row * a.ld_dx + col, n, pack8(dv, (const T*)nullptr));
    }
  }
  if (!a.dgamma && !a.dbeta) return;
  const bool alone = gridDim.x == 1;
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    float(&acc)[NV][8] = part ? db : dg;
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[sub][8 * (i * NT + t) + j] = acc[i][j];
      __syncthreads();
    }
    void* own = part ? a.dbeta : a.dgamma;
    float* to = a.part + (int64_t(blockIdx.x) * 2 + part) * cols;
    if constexpr (RPB > 1) {
      for (int c = threadIdx.x; c < cols; c += WG) {
        float s = sums[0][c];
#pragma unroll
        for (int g = 1; g < RPB; ++g) s += sums[g][c];
        if (!alone) to[c] = s;
        else if (own) Elem<W>::store((W*)own + c, s);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = 8 * (i * NT + t) + j;
          if (c < cols) {
            if (!alone) to[c] = acc[i][j];
            else if (own) Elem<W>::store((W*)own + c, acc[i][j]);
          }
        }
    }
  }
}

// Sums the workgroups' partial dgamma (blockIdx.y == 0) and dbeta over
// `parts` <= 512: 32 columns a workgroup, 32 slices of the parts, whose at
// most 16 loads are all in flight at once; the slices are joined in order.
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

constexpr int kFwdGrid = 2048;

template <typename T, typename W, bool FUSED> struct NormLaunch {
  template <int NT, int NV> static void fwd(const NormFwdArgs& a, hipStream_t st) {
    constexpr int WG = NT < 256 ? 256 : NT;
    const int64_t need = (a.rows + WG / NT - 1) / (WG / NT);
    hipLaunchKernelGGL((norm_fwd_kernel<T, W, NT, NV, WG, FUSED>), dim3(unsigned(std::min<int64_t>(need, kFwdGrid))),
                       dim3(WG), 0, st, a);
  }
  template <int NT, int NV, int WG> static void bwd(const NormBwdArgs& a, hipStream_t st) {
    const int64_t parts = norm_bwd_parts(a.rows, a.cols);
    hipLaunchKernelGGL((norm_bwd_kernel<T, W, NT, NV, WG, FUSED>), dim3(unsigned(parts)), dim3(WG), 0, st, a);
    if (parts > 1 && (a.dgamma || a.dbeta))
      hipLaunchKernelGGL((norm_grad_kernel<W>), dim3(unsigned((a.cols + kGradCols - 1) / kGradCols), 2),
                         dim3(kGradCols * kGradSlices), 0, st, a.part, int(parts), a.cols, (W*)a.dgamma, (W*)a.dbeta);
  }
  static hipError_t fwd(const NormFwdArgs& a, hipStream_t st) {
    switch (norm_row_threads(a.cols)) {
      case 16: fwd<16, 1>(a, st); break;
      case 64: a.cols <= 512 ? fwd<64, 1>(a, st) : fwd<64, 2>(a, st); break;
      case 256: a.cols <= 2048 ? fwd<256, 1>(a, st) : fwd<256, 2>(a, st); break;
      case 512: fwd<512, 2>(a, st); break;
      default: a.cols <= 16384 ? fwd<1024, 2>(a, st) : fwd<1024, 4>(a, st); break;
    }
    return hipGetLastError();
  }
  static hipError_t bwd(const NormBwdArgs& a, hipStream_t st) {
    switch (norm_row_threads(a.cols)) {
      case 16: bwd<16, 1, 512>(a, st); break;
      case 64: a.cols <= 512 ? bwd<64, 1, 512>(a, st) : bwd<64, 2, 512>(a, st); break;
      case 256: a.cols <= 2048 ? bwd<256, 1, 512>(a, st) : bwd<256, 2, 512>(a, st); break;
      case 512: bwd<512, 2, 512>(a, st); break;
      default: a.cols <= 16384 ? bwd<1024, 2, 1024>(a, st) : bwd<1024, 4, 1024>(a, st); break;
    }
    return hipGetLastError();
  }
};

template <typename A, typename F> hipError_t by_types(const A& a, bool bf16, bool wbf16, bool fused, F f) {
  auto go = [&](auto t, auto w) {
    typedef decltype(t) T;
    typedef decltype(w) W;
    return fused ? f(NormLaunch<T, W, true>{}) : f(NormLaunch<T, W, false>{});
  };
  if (bf16) return wbf16 ? go(uint16_t{}, uint16_t{}) : go(uint16_t{}, float{});
  return wbf16 ? go(float{}, uint16_t{}) : go(float{}, float{});
}

}  // namespace

hipError_t run_norm_fwd(const NormFwdArgs& a, bool bf16, bool wbf16, bool fused, hipStream_t st) {
  return by_types(a, bf16, wbf16, fused, [&](auto l) { return l.fwd(a, st); });
}

hipError_t run_norm_bwd(const NormBwdArgs& a, bool bf16, bool wbf16, bool fused, hipStream_t st) {
  return by_types(a, bf16, wbf16, fused, [&](auto l) { return l.bwd(a, st); });
}

}  // namespace muon
