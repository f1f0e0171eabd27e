// Device helpers of the training operators: 8-element vector access at any
// element alignment, reductions over lane groups, and the dropout generator.
#pragma once

#include "common.hpp"
#include "ops.hpp"

namespace muon {

// ---- 8 consecutive elements --------------------------------------------------
// gfx950 loads and stores 16 bytes at any address in global memory, so rows of
// odd width or stride take the same 16-byte accesses as aligned ones; only
// the end of a row that does not fill a vector goes in runs of 4, 2 and 1
// elements (three branches: a ladder of single elements made the compiler
// keep its masks and spill).
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_u __attribute__((aligned(2)));
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2_u __attribute__((ext_vector_type(2), aligned(4)));

template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> { u32x4 w; };
template <> struct Raw8<float> { f32x4 a, b; };

// The first n (any n, also <= 0 or > 8) of 8 elements at p; 0 in the others.
__device__ __forceinline__ Raw8<uint16_t> load8(const uint16_t* p, int n) {
  Raw8<uint16_t> r;
  r.w = u32x4{0, 0, 0, 0};
  if (n >= 8) {
    r.w = *(const u32x4_u*)p;
  } else if (n > 0) {
    u32x2 four{0, 0};
    uint32_t two = 0, one = 0;
    if (n & 4) four = *(const u32x2_u*)p;
    if (n & 2) two = *(const u32_u*)(p + (n & 4));
    if (n & 1) one = p[n & 6];
    const uint32_t t0 = (n & 2) ? two : one, t1 = (n & 2) ? one : 0;
    r.w = (n & 4) ? u32x4{four[0], four[1], t0, t1} : u32x4{t0, t1, 0, 0};
  }
  return r;
}
__device__ __forceinline__ Raw8<float> load8(const float* p, int n) {
  Raw8<float> r;
  r.a = f32x4{0, 0, 0, 0};
  r.b = f32x4{0, 0, 0, 0};
  if (n >= 8) {
    r.a = *(const f32x4_u*)p;
    r.b = *(const f32x4_u*)(p + 4);
  } else if (n > 0) {
    f32x2 two{0, 0};
    float one = 0;
    if (n & 4) r.a = *(const f32x4_u*)p;
    if (n & 2) two = *(const f32x2_u*)(p + (n & 4));
    if (n & 1) one = p[n & 6];
    const f32x4 t = (n & 2) ? f32x4{two[0], two[1], one, 0} : f32x4{one, 0, 0, 0};
    if (n & 4) r.b = t;
    else r.a = t;
  }
  return r;
}

// A row's vector at col, n = cols - col (0 in dead rows) of its 8 elements
// existing.  The last partial vector of a row is read as the row's last 8
// elements, in one access that waits for nothing, and settle8, called where
// the values are used, moves them to their places: with load8 the runs that
// make up a partial vector are waited for one after the other, which at 20000 x
// 1537 bf16 made the norm's backward pass 58.8 us instead of 53.6 (38.7 at 1536
// columns).
template <typename T>
__device__ __forceinline__ Raw8<T> load_row8(const T* row, unsigned col, int n, int cols) {
  if (cols < 8) return load8(row + col, n);
  if (n > 0 && n < 8) col = unsigned(cols - 8);
  return load8(row + col, n > 0 ? 8 : 0);
}
__device__ __forceinline__ void settle8(Raw8<uint16_t>& r, int n, int cols) {
  if (n > 0 && n < 8 && cols >= 8) {
    const int k = 8 - n;  // places to move down
    u32x4 w = r.w;
    w = (k & 4) ? u32x4{w[2], w[3], 0, 0} : w;
    w = (k & 2) ? u32x4{w[1], w[2], w[3], 0} : w;
    w = (k & 1) ? u32x4{w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, w[3] >> 16} : w;
    r.w = w;
  }
}
__device__ __forceinline__ void settle8(Raw8<float>& r, int n, int cols) {
  if (n > 0 && n < 8 && cols >= 8) {
    const int k = 8 - n;
    f32x4 a = r.a, b = r.b;
    const f32x4 zero{0, 0, 0, 0};
    if (k & 4) {
      a = b;
      b = zero;
    }
    if (k & 2) {
      a = f32x4{a[2], a[3], b[0], b[1]};
      b = f32x4{b[2], b[3], 0, 0};
    }
    if (k & 1) {
      a = f32x4{a[1], a[2], a[3], b[0]};
      b = f32x4{b[1], b[2], b[3], 0};
    }
    r.a = a;
    r.b = b;
  }
}

__device__ __forceinline__ void unpack8(const Raw8<uint16_t>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = r.a[i];
    v[4 + i] = r.b[i];
  }
}

// One rounding to the stored type (none for fp32).
__device__ __forceinline__ Raw8<uint16_t> pack8(const float (&v)[8], const uint16_t*) {
  Raw8<uint16_t> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] = f2bf2(v[2 * i], v[2 * i + 1]);
  return r;
}
__device__ __forceinline__ Raw8<float> pack8(const float (&v)[8], const float*) {
  Raw8<float> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.a[i] = v[i];
    r.b[i] = v[4 + i];
  }
  return r;
}

__device__ __forceinline__ void store8(uint16_t* p, int n, const Raw8<uint16_t>& r) {
  if (n >= 8) {
    *(u32x4_u*)p = r.w;
  } else if (n > 0) {
    uint32_t t0 = r.w[0], t1 = r.w[1];
    if (n & 4) {
      *(u32x2_u*)p = u32x2{t0, t1};
      t0 = r.w[2];
      t1 = r.w[3];
    }
    if (n & 2) {
      *(u32_u*)(p + (n & 4)) = t0;
      t0 = t1;
    }
    if (n & 1) p[n & 6] = uint16_t(t0);
  }
}
__device__ __forceinline__ void store8(float* p, int n, const Raw8<float>& r) {
  if (n >= 8) {
    *(f32x4_u*)p = r.a;
    *(f32x4_u*)(p + 4) = r.b;
  } else if (n > 0) {
    f32x4 t = r.a;
    if (n & 4) {
      *(f32x4_u*)p = t;
      t = r.b;
    }
    float one = t[0];
    if (n & 2) {
      *(f32x2_u*)(p + (n & 4)) = f32x2{t[0], t[1]};
      one = t[2];
    }
    if (n & 1) p[n & 6] = one;
  }
}

// 16 bytes of an output, past the caches if it is a stream (see kStreamOut).  The
// empty statements keep the compiler from making one ordinary store of the two.
__device__ __forceinline__ void put16(void* p, const u32x4& w, bool stream) {
  if (stream) {
    asm volatile("" ::: "memory");
    __builtin_nontemporal_store(w, (u32x4_u*)p);
    asm volatile("" ::: "memory");
  } else {
    *(u32x4_u*)p = w;
  }
}

// 16 bytes of a row: what a lane reads and writes at a time, so that a wave's
// accesses are adjacent in either type.
template <typename T> struct Piece;
template <> struct Piece<uint16_t> {
  static constexpr int N = 8;
  Raw8<uint16_t> r;
  template <bool STREAM> __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if (STREAM && n >= 8) r.w = __builtin_nontemporal_load((const u32x4_u*)p);
    else r = load8(p, n);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack8(r, v); }
  static __device__ __forceinline__ void store(uint16_t* p, int n, const float (&v)[8], bool stream) {
    const Raw8<uint16_t> w = pack8(v, p);
    if (n >= 8) put16(p, w.w, stream);
    else store8(p, n, w);
  }
};
template <> struct Piece<float> {
  static constexpr int N = 4;
  f32x4 r;
  template <bool STREAM> __device__ __forceinline__ void load(const float* p, int n) {
    r = f32x4{0, 0, 0, 0};
    if (n >= 4) {
      r = STREAM ? __builtin_nontemporal_load((const f32x4_u*)p) : *(const f32x4_u*)p;
    } else if (n > 0) {
      f32x2 two{0, 0};
      float one = 0;
      if (n & 2) two = *(const f32x2_u*)p;
      if (n & 1) one = p[n & 2];
      r = (n & 2) ? f32x4{two[0], two[1], one, 0} : f32x4{one, 0, 0, 0};
    }
  }
  __device__ __forceinline__ void get(float (&v)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = r[j];
  }
  static __device__ __forceinline__ void store(float* p, int n, const float (&v)[4], bool stream) {
    if (n >= 4) {
      put16(p, __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}), stream);
    } else if (n > 0) {
      if (n & 2) *(f32x2_u*)p = f32x2{v[0], v[1]};
      if (n & 1) p[n & 2] = v[n & 2];
    }
  }
};

// ---- reductions over groups of N adjacent lanes ---------------------------------
// Every lane of the group ends with the result; the order of the operations
// is fixed by the lane pattern.  Within 16 lanes by DPP (quad_perm, then
// mirrors: once a quad holds one value, mirroring 8 or 16 lanes pairs the
// quads), across them by the gfx950 row and half-wave swaps.
template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(x), CTRL, 0xf, 0xf, true));
}

template <int N, typename V, typename F> __device__ __forceinline__ V lane_reduce(V v, F f) {
  static_assert(sizeof(V) == 4 && (N == 4 || N == 8 || N == 16 || N == 32 || N == 64));
  auto bits = [](V x) { return __builtin_bit_cast(uint32_t, x); };
  auto val = [](uint32_t x) { return __builtin_bit_cast(V, x); };
  v = f(v, val(dpp<0xB1>(bits(v))));   // quad_perm [1,0,3,2]
  v = f(v, val(dpp<0x4E>(bits(v))));   // quad_perm [2,3,0,1]
  if constexpr (N >= 8) v = f(v, val(dpp<0x141>(bits(v))));   // mirror of 8 lanes
  if constexpr (N >= 16) v = f(v, val(dpp<0x140>(bits(v))));  // mirror of 16 lanes
  if constexpr (N >= 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(bits(v), bits(v), false, false);
    v = f(val(a[0]), val(a[1]));
  }
  if constexpr (N == 64) {
    const auto b = __builtin_amdgcn_permlane32_swap(bits(v), bits(v), false, false);
    v = f(val(b[0]), val(b[1]));
  }
  return v;
}
template <int N> __device__ __forceinline__ float lane_sum(float v) {
  return lane_reduce<N>(v, [](float a, float b) { return a + b; });
}

// Sum over the lanes that stand at the same place of their group of
// LANES.
template <int LANES> __device__ __forceinline__ float across_groups(float v) {
  if constexpr (LANES <= 8) v += __uint_as_float(dpp<0x128>(__float_as_uint(v)));  // 8 lanes on within 16
  if constexpr (LANES == 4) v += __uint_as_float(dpp<0x124>(__float_as_uint(v)));  // 4 lanes on within 16
  if constexpr (LANES <= 16) {
    const uint32_t x = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  if constexpr (LANES <= 32) {
    const uint32_t y = __float_as_uint(v);
    const auto b = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    v = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  }
  return v;
}

// ---- dropout's generator -------------------------------------------------------
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64 bit products, keyed
// by the seed.  The counter is (column / 8, row, offset): element c of a row
// takes halfword c % 8 of the 128 bits, low half of each word first, so the
// mask of an element depends on nothing but (seed, offset, row, column) and
// is formed again wherever it is needed.
__device__ __forceinline__ u32x4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                        uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
    const uint32_t n0 = uint32_t(b >> 32) ^ c1 ^ k0, n2 = uint32_t(a >> 32) ^ c3 ^ k1;
    c1 = uint32_t(b);
    c3 = uint32_t(a);
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

__device__ __forceinline__ uint64_t drop_offset(const DropArgs& d) {
  return d.offset + (d.offset_dev ? *d.offset_dev : 0);
}

// The 8 draws of one vector.
__device__ __forceinline__ u32x4 drop_draws(const DropArgs& d, uint64_t off, uint32_t row, uint32_t block) {
  return philox(block, row, uint32_t(off), uint32_t(off >> 32), d.k0, d.k1);
}
__device__ __forceinline__ bool drop_keeps(const u32x4& w, int i, uint32_t thresh) {
  return ((i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu) >= thresh;
}

}  // namespace muon
