// Row-wise building blocks of the loss and norm kernels: eight consecutive
// elements per lane and access, exponentials, and sums across lanes.
//
// Rows may start at any element: the 16-byte accesses go through
// __builtin_memcpy with the element's own alignment, which this target turns
// into one global_load/store_dwordx4 (its global memory accesses need no
// alignment), so odd widths and odd strides take the same path.
#pragma once

#include "common.hpp"

namespace detgrad {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Element types: uint16_t holds bf16 bits, float is float32.
__device__ __forceinline__ float to_f32(uint16_t b) { return bf16_to_f32(b); }
__device__ __forceinline__ float to_f32(float f) { return f; }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
// bf16 by round to nearest even, NaN kept (the target's conversion instruction)
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// Eight elements as they are in memory (16 bytes of bf16, 32 of float32).
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  u32x4 w;
  __device__ __forceinline__ void load(const uint16_t* p) { __builtin_memcpy(&w, p, 16); }
  __device__ __forceinline__ void load_short(const uint16_t* p, int n) {  // n in [1, 8): the last element repeats
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = static_cast<uint32_t>(p[2 * i < n ? 2 * i : n - 1]) |
             (static_cast<uint32_t>(p[2 * i + 1 < n ? 2 * i + 1 : n - 1]) << 16);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  }
};
template <>
struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    __builtin_memcpy(&a, p, 16);
    __builtin_memcpy(&b, p + 4, 16);
  }
  __device__ __forceinline__ void load_short(const float* p, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = p[i < n ? i : n - 1];
      b[i] = p[i + 4 < n ? i + 4 : n - 1];
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
};

// v = the elements p[0..7]; those at or past n (n <= 0: all of them) are `fill`
// and are not read.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t n, float fill, float (&v)[8]) {
  if (n >= 8) {
    Raw8<T> r;
    r.load(p);
    r.get(v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : fill;
  }
}

// In a block under a condition that is the same for all lanes and seldom true:
// keeps the compiler from computing the block always and selecting.
__device__ __forceinline__ void keep_branch() { asm volatile(""); }

// Stores of eight elements. PAST: past the caches, for outputs larger than they
// are: their reader would not find them there anyway, and their dirty lines
// would be written back among other reads.
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
template <bool PAST>
__device__ __forceinline__ void store8_full(float* p, const float (&v)[8]) {
  const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
  if constexpr (PAST) {
    __builtin_nontemporal_store(a, reinterpret_cast<f32x4_a4*>(p));
    __builtin_nontemporal_store(b, reinterpret_cast<f32x4_a4*>(p + 4));
  } else {
    __builtin_memcpy(p, &a, 16);
    __builtin_memcpy(p + 4, &b, 16);
  }
}
template <bool PAST>
__device__ __forceinline__ void store8_full(uint16_t* p, const float (&v)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(from_f32<uint16_t>(v[2 * i])) |
           (static_cast<uint32_t>(from_f32<uint16_t>(v[2 * i + 1])) << 16);
  if constexpr (PAST)
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4_a2*>(p));
  else
    __builtin_memcpy(p, &w, 16);
}

// p[0..min(n, 8)) = v, rounded once to the element type.
template <typename T>
__device__ __forceinline__ void store8(T* p, int64_t n, const float (&v)[8]) {
  if (n >= 8) {
    store8_full<false>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

// A lane's eight columns of rows of N elements, chosen so that the lane's load is
// one unconditional access inside the row (loads under a branch would be waited
// for one by one): columns base .. base + 7, of which those in [lo, hi) are the
// lane's own. The lane that would cross the row's end moves back to N - 8 and
// leaves the columns it shares with its neighbour alone; a lane past the end
// (lo = 8) owns none and reads the row's start. Rows of N < 8 elements, which
// only instances with TINY meet, are loaded element by element.
template <bool TINY>
struct Cols {
  int base, lo, hi;
  bool all;  // every lane of the launch owns eight columns (the same everywhere)
  __device__ __forceinline__ bool own(int j) const { return j >= lo && (!TINY || j < hi); }
  // col: the lane's first column, a multiple of 8; cover: the columns of all lanes
  __device__ __forceinline__ void set(int col, int N, int cover) {
    all = N == cover;
    hi = TINY && N < 8 ? N : 8;
    base = col + 8 <= N ? col : (col < N && hi == 8 ? N - 8 : 0);
    lo = col < N ? col - base : 8;
  }
};
template <typename T, bool TINY>
__device__ __forceinline__ void load_cols(Raw8<T>& r, const T* row, const Cols<TINY>& c) {
  if (TINY && c.hi < 8)  // (the same for every lane)
    r.load_short(row, c.hi);
  else
    r.load(row + c.base);
}
// v = the loaded values, `fill` in columns that are not the lane's own
template <typename T, bool TINY>
__device__ __forceinline__ void get_cols(const Raw8<T>& r, const Cols<TINY>& c, float fill, float (&v)[8]) {
  r.get(v);
  if (!c.all) {
    keep_branch();
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c.own(j) ? v[j] : fill;
  }
}
template <bool PAST = false, typename T, bool TINY>
__device__ __forceinline__ void store_cols(T* row, const Cols<TINY>& c, const float (&v)[8]) {
  if (c.all || (c.lo == 0 && (!TINY || c.hi == 8))) {
    store8_full<PAST>(row + c.base, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c.own(j)) row[c.base + j] = from_f32<T>(v[j]);
  }
}

constexpr float kLog2e = 0x1.715476p+0f, kLog2eLo = 0x1.4ae0c0p-26f, kLn2 = 0x1.62e430p-1f;

// exp(x) within about 1.5 units in the last place: x log2(e) = k + f with k
// whole, f from two fused steps against a two-word log2(e) (so the reduction's
// error does not grow with |x|), then the hardware's 2^f scaled by 2^k.
// exp(-inf) = 0, NaN stays NaN, results below 2^-149 are 0.
__device__ __forceinline__ float exp_e(float x) {
  const float k = __builtin_rintf(x * kLog2e);
  const float f = __builtin_fmaf(x, kLog2eLo, __builtin_fmaf(x, kLog2e, -k));
  const float y = __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), static_cast<int>(k));
  return x < -104.0f ? 0.0f : (x > 89.0f ? __builtin_inff() : y);
}

// The lane swaps of a value with itself give every lane the copies of both
// partners at distance 16 or 32 (a from the lower, b from the upper), on the
// VALU instead of through LDS; every lane of the wave must be active.
struct Halves {
  float a, b;
};
__device__ __forceinline__ Halves halves16(float v) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return {__uint_as_float(p[0]), __uint_as_float(p[1])};
}
__device__ __forceinline__ Halves halves32(float v) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return {__uint_as_float(p[0]), __uint_as_float(p[1])};
}

// Sum / maximum over groups of W consecutive lanes (W a power of two); every
// lane of a group ends with the group's value, added in one fixed tree.
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (W >= 2) v = v + dpp_mov<DPP_XOR1>(v);
  if constexpr (W >= 4) v = v + dpp_mov<DPP_XOR2>(v);
  if constexpr (W >= 8) v = v + dpp_mov<DPP_HALF_MIRROR>(v);
  if constexpr (W >= 16) v = v + dpp_mov<DPP_MIRROR>(v);
  if constexpr (W >= 32) {
    const Halves h = halves16(v);
    v = h.a + h.b;
  }
  if constexpr (W >= 64) {
    const Halves h = halves32(v);
    v = h.a + h.b;
  }
  return v;
}
template <int W>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (W >= 2) v = fmaxf(v, dpp_mov<DPP_XOR1>(v));
  if constexpr (W >= 4) v = fmaxf(v, dpp_mov<DPP_XOR2>(v));
  if constexpr (W >= 8) v = fmaxf(v, dpp_mov<DPP_HALF_MIRROR>(v));
  if constexpr (W >= 16) v = fmaxf(v, dpp_mov<DPP_MIRROR>(v));
  if constexpr (W >= 32) {
    const Halves h = halves16(v);
    v = fmaxf(h.a, h.b);
  }
  if constexpr (W >= 64) {
    const Halves h = halves32(v);
    v = fmaxf(h.a, h.b);
  }
  return v;
}

// ------------------------------------------------------------------ host side
// Size of the last-level cache: calls whose outputs together reach it store them
// past the caches. Measured with the distillation: a step at 4096 x 32768 bf16
// (256 MiB of dz) 142 us against 169 with ordinary stores. Smaller outputs are 5 % faster to store that way as well,
// but the kernel that reads them next loses more: at 128 MiB of dz 3 us gained, 37
// lost by a reduction over dz that took 295.
constexpr int64_t kCacheBytes = int64_t(256) << 20;
inline bool past_caches(int64_t out_bytes) { return out_bytes >= kCacheBytes; }

// One buffer of a call, the size of its elements, and for rows with a stride the
// bytes of a row and from row to row (0: one piece).
struct Buf {
  const char* name;
  Range r;
  size_t elem = 4, width = 0, pitch = 0;
};
inline Buf buf_rows(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, size_t elem) {
  return {name, range2d(p, rows, cols, ld, elem), elem, static_cast<size_t>(cols) * elem, static_cast<size_t>(ld) * elem};
}

// Whether two buffers share a byte. Rows with one stride that take different
// columns of it (two halves of one [T, 2D] buffer) lie between each other; for
// other strides the spans decide.
inline bool overlaps(const Buf& a, const Buf& b) {
  if (!overlaps(a.r, b.r)) return false;
  if (a.pitch == 0 || a.pitch != b.pitch) return true;
  const size_t d = a.r.lo <= b.r.lo ? (b.r.lo - a.r.lo) % a.pitch : (a.pitch - (a.r.lo - b.r.lo) % a.pitch) % a.pitch;
  return d < a.width || d + b.width > a.pitch;
}

// Every buffer starts on a border of its element type, and no output overlaps an
// input, another output or the workspace.
inline int check_buffers(const char* what, const Buf* outs, int n_out, const Buf* ins, int n_in) {
  for (int i = 0; i < n_out + n_in; ++i) {
    const Buf& b = i < n_out ? outs[i] : ins[i - n_out];
    if (b.r.lo % b.elem)
      return set_error(DET_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", what, b.name);
  }
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlaps(outs[i], ins[j]))
        return set_error(DET_ERR_OVERLAP, "%s: %s overlaps %s", what, outs[i].name, ins[j].name);
    for (int j = i + 1; j < n_out; ++j)
      if (overlaps(outs[i], outs[j]))
        return set_error(DET_ERR_OVERLAP, "%s: %s overlaps %s", what, outs[i].name, outs[j].name);
  }
  return DET_OK;
}

inline int check_float_dtype(const char* what, int dtype) {
  if (dtype != DET_BF16 && dtype != DET_F32)
    return set_error(DET_ERR_INVALID_ARG, "%s: dtype must be DET_BF16 or DET_F32, got %d", what, dtype);
  return DET_OK;
}
inline size_t dtype_size(int dtype) { return dtype == DET_BF16 ? 2 : 4; }

}  // namespace detgrad
