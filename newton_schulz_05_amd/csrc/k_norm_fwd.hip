// Layer norm, forward (see norm_dev.hpp).
#include "norm_dev.hpp"

namespace muon {

namespace {

// Bound by memory: x is read and y written once (16384 x 4096 bf16: 51.5
// us, 5.2 TB/s, the rate of a large copy).  gamma and beta come from the cache, their loads
// behind those of x; with three and more vectors a thread they are read after
// the reductions, over which they would take registers.
template <typename T, typename W, int NT, int NV, int WG, bool FUSED, bool RAG>
__global__ __launch_bounds__(WG) void norm_fwd_kernel(NormFwdArgs a) {
  constexpr int RPB = WG / NT;
  constexpr bool EARLY = NV <= 2;
  __shared__ float red[4][WG / 64], pair[WG / 64][2];
  const int t = threadIdx.x % NT, sub = row_group<NT>();
  const int cols = a.cols;
  const uint64_t off = FUSED ? drop_offset(a.drop) : 0;
  for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < a.rows; row0 += int64_t(gridDim.x) * RPB) {
    const int64_t row = row0 + sub;
    const bool live = row < a.rows;
    Raw8<T> xr[NV], rr[NV];
    Raw8<W> gr[NV], br[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const unsigned col = 8 * (i * NT + t);
      const int n = live ? cols - int(col) : 0;
      xr[i] = load_vec<RAG>((const T*)a.x + row * a.ld_x, col, n, a.cols);
      if constexpr (FUSED) rr[i] = load_vec<RAG>((const T*)a.res + row * a.ld_res, col, n, a.cols);
    }
    if constexpr (EARLY) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const unsigned col = 8 * (i * NT + t);
        gr[i] = load_param<RAG, W>(a.gamma, col, cols);
        br[i] = load_param<RAG, W>(a.beta, col, cols);
      }
    }
    float v[NV][8];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const unsigned col = 8 * (i * NT + t);
      const int n = live ? cols - int(col) : 0;
      settle<RAG>(xr[i], n, cols);
      unpack8(xr[i], v[i]);
      if constexpr (FUSED) {
        float rv[8];
        settle<RAG>(rr[i], n, cols);
        unpack8(rr[i], rv);
        const u32x4 w = drop_draws(a.drop, off, uint32_t(row), col / 8);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i][j] = drop_keeps(w, j, a.drop.thresh) ? fmaf(v[i][j], a.drop.scale, rv[j]) : rv[j];
        // the norm is that of h as it is stored, so that the backward pass,
        // which reads h, sees the same values
        const Raw8<T> hr = pack8(v[i], (const T*)nullptr);
        store_vec<RAG>((T*)a.h + row * a.ld_h + col, n, hr);
        unpack8(hr, v[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s += !RAG || j < n ? v[i][j] : 0.0f;  // 0 in a vector that does not exist
    }
    float mean = row_sum<NT>(s, red[0]) / float(cols);
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int n = cols - 8 * (i * NT + t);
      const float m = RAG || n > 0 ? mean : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] -= m;
        q = !RAG || j < n ? fmaf(v[i][j], v[i][j], q) : q;
      }
    }
    // The mean's roundings are of the size of the row's offset.  Where that is
    // more than two deviations, the mean of the deviations is taken off as well
    // and the squares are summed again (without this a constant row of 1000.1
    // gave y = 0.04 at 4096 columns); elsewhere the error is a few roundings of
    // the deviation.  A test of each row, not the same for all: two more
    // operations an element for every row cost 8 to 14 % of a pass out of the
    // cache (bf16 20000 x 1536, 65536 x 200).  The branch is taken together by
    // the threads that share its sums' lanes or barriers: with two rows a
    // workgroup each tests the other row as well.
    const float square = mean * mean * float(cols);
    bool offset, any;
    if constexpr (NT > 64 && RPB == 2) {
      constexpr int NW = NT / 64;
      const int wave = threadIdx.x / 64, own = wave / NW * NW, other = own ^ NW;
      q = lane_sum<64>(q);
      if (threadIdx.x % 64 == 0) {
        pair[wave][0] = q;
        pair[wave][1] = square;
      }
      __syncthreads();
      q = pair[own][0];
      float w = pair[other][0];
#pragma unroll
      for (int i = 1; i < NW; ++i) {
        q += pair[own + i][0];
        w += pair[other + i][0];
      }
      offset = !(square <= 4.0f * q);
      any = offset || !(pair[other][1] <= 4.0f * w);
    } else {
      static_assert(NT <= 64 || RPB == 1);
      q = row_sum<NT>(q, red[1]);
      offset = !(square <= 4.0f * q);
      any = NT > 64 ? offset : __any(offset);
    }
    if (any) {
      float d = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = cols - 8 * (i * NT + t);
#pragma unroll
        for (int j = 0; j < 8; ++j) d += j < n ? v[i][j] : 0.0f;
      }
      d = row_sum<NT>(d, red[2]) / float(cols);
      d = offset ? d : 0.0f;
      mean += d;
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = cols - 8 * (i * NT + t);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] -= d;
          s = j < n ? fmaf(v[i][j], v[i][j], s) : s;
        }
      }
      s = row_sum<NT>(s, red[3]);
      q = offset ? s : q;
    }
    const float rstd = 1.0f / sqrtf(q / float(cols) + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const unsigned col = 8 * (i * NT + t);
      const int n = live ? cols - int(col) : 0;
      if constexpr (!EARLY) {
        gr[i] = load_param<RAG, W>(a.gamma, col, cols);
        br[i] = load_param<RAG, W>(a.beta, col, cols);
      }
      float gv[8], bv[8];
      settle<RAG>(gr[i], cols - int(col), cols);
      settle<RAG>(br[i], cols - int(col), cols);
      unpack_param(gr[i], a.gamma, 1.0f, gv);
      unpack_param(br[i], a.beta, 0.0f, bv);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * rstd, gv[j], bv[j]);
      store_vec<RAG>((T*)a.y + row * a.ld_y + col, n, pack8(v[i], (const T*)nullptr));
    }
    if (live && t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

template <typename T, typename W, bool FUSED, bool RAG> struct FwdLaunch {
  // One group of rows a workgroup: new workgroups keep loads in flight while
  // others reduce (16384 x 4096 bf16: 51.5 us; 59.2 with the rows dealt to 2048
  // workgroups that loop, 66.0 to 512).
  template <int NT, int NV> static void fwd(const NormFwdArgs& a, hipStream_t st) {
    // 128 threads a row: two rows a workgroup, but one in the leanest kernels
    // (bf16 20000 x 1536 26.1 us with one, 27.4 with two, 60000 rows 66.7 and
    // 71.4; 1537 columns 38.9 and 38.0, fused 67.3 and 64.5; fp32 1536 columns
    // 53.3 and 49.9).
    constexpr int WG = NT == 128 && sizeof(T) == 2 && !FUSED && !RAG ? 128 : NT < 256 ? 256 : NT;
    const int64_t need = (a.rows + WG / NT - 1) / (WG / NT);
    hipLaunchKernelGGL((norm_fwd_kernel<T, W, NT, NV, WG, FUSED, RAG>), dim3(unsigned(std::min(need, kOpsMaxGrid))),
                       dim3(WG), 0, st, a);
  }
  static hipError_t fwd(const NormFwdArgs& a, hipStream_t st) {
    // The narrowest fit that keeps several workgroups on a compute unit: three
    // to five vectors a thread rather than 512 or 1024 threads a row (bf16 16384
    // x 8192: 98.5 us with 256 threads, 107.0 with 512; 3300 x 20000: 60.1 with
    // 512, 66.9 with 1024; 16384 x 2048: 26.9 with 128, 28.6 with 256; 65536 x
    // 200: 13.0 with 32, 22.0 with 64).
    const int vecs = (a.cols + 7) / 8;
    if (vecs <= 8) fwd<8, 1>(a, st);
    else if (vecs <= 16) fwd<16, 1>(a, st);
    else if (vecs <= 32) fwd<32, 1>(a, st);
    else if (vecs <= 64) fwd<64, 1>(a, st);
    else if (vecs <= 128) fwd<64, 2>(a, st);
    else if (vecs <= 256) fwd<128, 2>(a, st);
    else if (vecs <= 512) fwd<256, 2>(a, st);
    else if (vecs <= 768) fwd<256, 3>(a, st);
    else if (vecs <= 1024) fwd<256, 4>(a, st);
    else if (vecs <= 1280) fwd<256, 5>(a, st);
    else if (vecs <= 1536) fwd<512, 3>(a, st);
    else if (vecs <= 2048) fwd<512, 4>(a, st);
    else if (vecs <= 2560) fwd<512, 5>(a, st);
    else fwd<1024, 4>(a, st);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t run_norm_fwd(const NormFwdArgs& a, bool bf16, bool wbf16, bool fused, hipStream_t st) {
  return norm_by_types<FwdLaunch>(a.cols, bf16, wbf16, fused, [&](auto l) { return l.fwd(a, st); });
}

}  // namespace muon
