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
// A row is read once and held in registers by 8 to 1024 threads, so the mean
// (and for a row far off 0 the mean of the deviations from it) comes before the
// squared deviations are formed, without a second pass over memory.  All sums
// are fp32; each output is rounded once.
#pragma once

#include "ops_dev.hpp"

// Products and sums are joined only where fmaf says so, so that every variant
// of a kernel (fused or not, any row split) rounds alike.
#pragma clang fp contract(off)

namespace muon {

// Sum over the NT threads of a row; `red` holds one word per wave and row.
// Sums that follow one another take different `red` buffers, so that one
// barrier per sum is enough.
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

// Which of the workgroup's row groups a thread is in: the same for a whole
// wave from 64 threads a row on, so that row addresses stay in scalar
// registers (as lane values they spilled above 8192 columns).
template <int NT> __device__ __forceinline__ int row_group() {
  const int g = threadIdx.x / NT;
  return NT >= 64 ? __builtin_amdgcn_readfirstlane(g) : g;
}

// Vectors of a row at col, n = cols - col elements of it existing (0 in dead
// rows).  Without RAG cols is a multiple of 8, so that a vector exists whole or
// not at all; with it see load_row8.  (One code for both costs whole rows their
// tests of n and the shift: 20000 x 1536 bf16 forward 25.6 us without RAG, 37.9
// with; 16384 x 8192 backward 150.9 and 161.6.)
template <bool RAG, typename T>
__device__ __forceinline__ Raw8<T> load_vec(const T* row, unsigned col, int n, int cols) {
  if constexpr (RAG) return load_row8(row, col, n, cols);
  else return load8(row + col, n > 0 ? 8 : 0);
}
template <bool RAG, typename T> __device__ __forceinline__ void settle(Raw8<T>& r, int n, int cols) {
  if constexpr (RAG) settle8(r, n, cols);
}
template <bool RAG, typename T> __device__ __forceinline__ void store_vec(T* p, int n, const Raw8<T>& r) {
  store8(p, RAG ? n : (n > 0 ? 8 : 0), r);
}

// gamma or beta as stored; `dflt` in the place of a null one.
template <bool RAG, typename W>
__device__ __forceinline__ Raw8<W> load_param(const void* p, unsigned col, int cols) {
  return load_vec<RAG>((const W*)p, col, p ? cols - int(col) : 0, cols);
}
template <typename W>
__device__ __forceinline__ void unpack_param(const Raw8<W>& r, const void* p, float dflt, float (&v)[8]) {
  unpack8(r, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = p ? v[i] : dflt;
}

// Calls f with the launches for the call's types.
template <template <typename, typename, bool, bool> class Launch, typename F>
hipError_t norm_by_types(int cols, bool bf16, bool wbf16, bool fused, F f) {
  auto go = [&](auto t, auto w) {
    typedef decltype(t) T;
    typedef decltype(w) W;
    const bool rag = cols % 8 != 0;
    return fused ? (rag ? f(Launch<T, W, true, true>{}) : f(Launch<T, W, true, false>{}))
                 : (rag ? f(Launch<T, W, false, true>{}) : f(Launch<T, W, false, false>{}));
  };
  if (bf16) return wbf16 ? go(uint16_t{}, uint16_t{}) : go(uint16_t{}, float{});
  return wbf16 ? go(float{}, uint16_t{}) : go(float{}, float{});
}

}  // namespace muon
