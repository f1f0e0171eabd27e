// Dropout from a counter-based generator, with an optional residual add:
// out = residual + keep(seed, offset, row, column) * x / (1 - p).  The mask
// is formed from the counter wherever it is needed (the backward pass is the
// same call on the gradient), never stored, so the operator moves 2 (3 with
// the residual) times the tensor's bytes.
#include "ops_dev.hpp"

namespace muon {

namespace {

constexpr int kDropThreads = 256;

// Thread v of the grid takes vectors v, v + step, ... of 8 elements, counted
// row by row; the step is split into rows and vectors on the host, so that a
// thread divides once.
template <typename T, bool RES>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(DropoutArgs a, uint32_t per_row, uint32_t step_rows,
                                                               uint32_t step_vecs) {
  const uint64_t first = uint64_t(blockIdx.x) * kDropThreads + threadIdx.x;
  uint64_t row = uint32_t(first) / per_row;
  uint32_t vec = uint32_t(first) - uint32_t(row) * per_row;
  const uint64_t off = drop_offset(a.drop);
  while (row < uint64_t(a.rows)) {
    const int64_t col = int64_t(vec) * 8;
    const int n = a.cols - col >= 8 ? 8 : int(a.cols - col);
    // the row's end, as load_row8 takes it (columns here may pass 32 bits)
    const bool whole = a.cols >= 8;
    const int64_t at = whole ? (n < 8 ? a.cols - 8 : col) : col;
    const int take = whole ? 8 : n;
    float v[8], rv[8];
    Raw8<T> xr = load8((const T*)a.x + row * a.ld_x + at, take), rr;
    if constexpr (RES) rr = load8((const T*)a.res + row * a.ld_res + at, take);
    settle8(xr, n, take);
    unpack8(xr, v);
    if constexpr (RES) {
      settle8(rr, n, take);
      unpack8(rr, rv);
    }
    const u32x4 w = drop_draws(a.drop, off, uint32_t(row), vec);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool keep = drop_keeps(w, j, a.drop.thresh);
      if constexpr (RES) v[j] = keep ? fmaf(v[j], a.drop.scale, rv[j]) : rv[j];
      else v[j] = keep ? v[j] * a.drop.scale : 0.0f;
    }
    store8((T*)a.out + row * a.ld_out + col, n, pack8(v, (const T*)nullptr));
    row += step_rows;
    vec += step_vecs;
    if (vec >= per_row) {
      vec -= per_row;
      ++row;
    }
  }
}

template <typename T> void launch(const DropoutArgs& a, hipStream_t st) {
  const uint64_t per_row = uint64_t(a.cols + 7) / 8;
  // a lone long row and many short ones alike: enough workgroups for all
  // vectors, at most kOpsMaxGrid
  const uint64_t total = per_row * uint64_t(a.rows);
  const uint64_t grid = std::min<uint64_t>((total + kDropThreads - 1) / kDropThreads, uint64_t(kOpsMaxGrid));
  const uint64_t step = grid * kDropThreads;
  const uint32_t sr = uint32_t(step / per_row), sv = uint32_t(step % per_row);
  if (a.res)
    hipLaunchKernelGGL((dropout_kernel<T, true>), dim3(unsigned(grid)), dim3(kDropThreads), 0, st, a,
                       uint32_t(per_row), sr, sv);
  else
    hipLaunchKernelGGL((dropout_kernel<T, false>), dim3(unsigned(grid)), dim3(kDropThreads), 0, st, a,
                       uint32_t(per_row), sr, sv);
}

}  // namespace

hipError_t run_dropout(const DropoutArgs& a, bool bf16, hipStream_t st) {
  bf16 ? launch<uint16_t>(a, st) : launch<float>(a, st);
  return hipGetLastError();
}

}  // namespace muon
