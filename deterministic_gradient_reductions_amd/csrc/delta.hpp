// Building blocks of the gated delta rule's kernels: 16 x 16 tiles on the matrix
// cores with operands in one to three bf16 words, and their fragments in LDS.
//
// Words. A float32 x is carried into a product as x0 + x1 + x2, x0 = bf16(x), x1 =
// bf16(x - x0), x2 the rest (both differences are exact): 8 bits of it per word.
// bf16 inputs are one word and exact. A product of operands of NA and NB words sums
// the terms i + j < P; what is left out is 2^-9P of the operands. The instruction's
// own sums are float32. So v_mfma_f32_16x16x32_bf16 (16 times the rate of the
// float32 instruction) gives float32 products in six terms, and products of a bf16
// input with a float32 state in three.
//
// Layout. The instruction takes lane l = 16 g + c as row (A) or column (B) c of its
// operands with eight of the 32 places of the summed index, and gives it the rows
// 4 g + r (r = 0..3) of column c of the result. Which eight places a lane group g
// takes is free as long as A and B agree; here they are 4 g + r and 16 + 4 g + r.
// Then the results of two tiles, one below the other, are an operand of the next
// product as they stand, summed over their rows: a chain of products keeps its
// running operand in registers.
#pragma once

#include "rowops.hpp"
#include "segtiles.hpp"

namespace detgrad {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

template <int NP>
struct Frag {
  bf16x8 w[NP];
};

// acc += A B over the terms i + j < P, the smallest first.
template <int P, int NA, int NB>
__device__ __forceinline__ void mm(f32x4& acc, const Frag<NA>& a, const Frag<NB>& b) {
#pragma unroll
  for (int s = P - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.w[i], b.w[s - i], acc, 0, 0, 0);
}

template <int NP>
__device__ __forceinline__ void split(float x, __bf16 (&w)[NP]) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    w[p] = static_cast<__bf16>(x);
    if (p + 1 < NP) x -= static_cast<float>(w[p]);
  }
}

// The fragment whose places are the rows of two results, x above y.
template <int NP>
__device__ __forceinline__ Frag<NP> frag_of(const f32x4& x, const f32x4& y) {
  Frag<NP> f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    __bf16 a[NP], b[NP];
    split<NP>(x[r], a);
    split<NP>(y[r], b);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      f.w[p][r] = a[p];
      f.w[p][4 + r] = b[p];
    }
  }
  return f;
}

// Fragments of an operand of 16 RT rows (or columns) and 32 KS places in LDS, NP
// words. A lane's 16 bytes lie side by side for the 16 rows; the lane groups are 272
// bytes apart and the row tiles a multiple of 256 bytes and 16 more, so that the
// 8-byte writes of four neighbouring places, rows or columns running over the
// lanes, spread over the banks.
template <int RT, int KS, int NP>
struct Image {
  static constexpr int kGroup = 272, kFrag = 4 * kGroup, kTile = (KS * kFrag + 239) / 256 * 256 + 16, kWord = RT * kTile;
  static constexpr int kBytes = NP * kWord;
  static_assert(kTile >= KS * kFrag && kTile % 16 == 0, "tiles overlap");
  // row (16 rt + c), places 32 ks + 16 half + 4 g .. + 3
  static __device__ __forceinline__ int at(int row, int place) {
    return (row >> 4) * kTile + (place >> 5) * kFrag + ((place >> 2) & 3) * kGroup + (row & 15) * 16 + ((place >> 4) & 1) * 8;
  }
  static __device__ __forceinline__ Frag<NP> load(const char* base, int rt, int ks) {
    const int lane = threadIdx.x & 63;
    Frag<NP> f;
#pragma unroll
    for (int p = 0; p < NP; ++p)
      f.w[p] = *reinterpret_cast<const bf16x8*>(base + p * kWord + rt * kTile + ks * kFrag + (lane >> 4) * kGroup +
                                                (lane & 15) * 16);
    return f;
  }
  // the places place .. place + 3 (place a multiple of 4) of a row
  static __device__ __forceinline__ void store4(char* base, int row, int place, const float (&v)[4]) {
    bf16x4 w[NP];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __bf16 x[NP];
      split<NP>(v[j], x);
#pragma unroll
      for (int p = 0; p < NP; ++p) w[p][j] = x[p];
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) *reinterpret_cast<bf16x4*>(base + p * kWord + at(row, place)) = w[p];
  }
  static __device__ __forceinline__ void store1(char* base, int row, int place, float v) {
    __bf16 x[NP];
    split<NP>(v, x);
#pragma unroll
    for (int p = 0; p < NP; ++p)
      *reinterpret_cast<__bf16*>(base + p * kWord + at(row, place & ~3) + (place & 3) * 2) = x[p];
  }
};

// Four consecutive elements, those at or past n zero (and not read).
template <typename T>
struct Raw4;
template <>
struct Raw4<uint16_t> {
  uint32_t a, b;
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    a = b = 0;
    if (n >= 4) {
      uint64_t w;
      __builtin_memcpy(&w, p, 8);
      a = static_cast<uint32_t>(w);
      b = static_cast<uint32_t>(w >> 32);
    } else if (n > 0) {
      a = p[0] | (n > 1 ? static_cast<uint32_t>(p[1]) << 16 : 0u);
      b = n > 2 ? p[2] : 0u;
    }
  }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = bf16_lo(a);
    v[1] = bf16_hi(a);
    v[2] = bf16_lo(b);
    v[3] = bf16_hi(b);
  }
};
template <>
struct Raw4<float> {
  f32x4 w;
  __device__ __forceinline__ void load(const float* p, int n) {
    w = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (n >= 4) {
      __builtin_memcpy(&w, p, 16);
    } else {
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (j < n) w[j] = p[j];
    }
  }
  __device__ __forceinline__ void get(float (&v)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = w[j];
  }
};
// p[0 .. min(n, 4)) = v, rounded once
__device__ __forceinline__ void store4(float* p, int n, const f32x4& v) {
  if (n >= 4) {
    __builtin_memcpy(p, &v, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < n) p[j] = v[j];
  }
}
__device__ __forceinline__ void store4(uint16_t* p, int n, const f32x4& v) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = static_cast<uint32_t>(from_f32<uint16_t>(v[2 * i])) |
           (static_cast<uint32_t>(from_f32<uint16_t>(v[2 * i + 1])) << 16);
  if (n >= 4) {
    __builtin_memcpy(p, w, 8);
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < n) p[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
  }
}

// Writes to LDS of this wave's lanes are seen by its other lanes after this (the
// wave's LDS accesses run in order; the compiler must not reorder them).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A [T, heads, dim] tensor with unit innermost stride.
template <typename T>
struct Heads {
  T* p;
  int64_t st, sh;
  __device__ __forceinline__ T* row(int64_t t, int h) const { return p + t * st + h * sh; }
};

// Rows [r0, r1) of segment s and the tiles before it, from the clamped offsets (see
// segment_tile); every lane of the wave active.
__device__ __forceinline__ void segment_rows(const int32_t* __restrict__ offs, int s, uint32_t M, int log_bm, uint32_t& r0,
                                             uint32_t& r1, uint32_t& first) {
  const int lane = threadIdx.x & 63;
  const uint32_t bm = 1u << log_bm;
  uint32_t run_b = clamp_off(offs[0], M), run_t = 0;
  for (int e0 = 0;; e0 += 64) {
    const int e = e0 + lane;
    const uint32_t b1 = umax(scan_max(clamp_off(offs[e <= s ? e + 1 : s + 1], M)), run_b);
    const uint32_t b0 = from_lane_below(b1, run_b);
    const uint32_t nt = e <= s && b1 > b0 ? (b1 - b0 + bm - 1) >> log_bm : 0u;
    const uint32_t incl = scan_add(nt);
    if (s < e0 + 64) {
      r0 = lane_value(b0, s - e0);
      r1 = lane_value(b1, s - e0);
      first = run_t + lane_value(incl - nt, s - e0);
      return;
    }
    run_t += lane_value(incl, 63);
    run_b = lane_value(b1, 63);
  }
}

// Tokens per chunk, words of an input, words of what only reaches outputs of the
// input's type. float32 takes half the chunk: its images have three words.
template <typename T>
struct DeltaType;
template <>
struct DeltaType<uint16_t> {
  static constexpr int kLogC = 6, kIn = 1, kOut = 2;
};
template <>
struct DeltaType<float> {
  static constexpr int kLogC = 5, kIn = 3, kOut = 3;
};
// Words of what reaches a float32 state, whose errors stay.
constexpr int kStateWords = 3;

// What the preparing kernel leaves per (chunk, value head): the inverse [C][C] (its
// tiles above the diagonal are not written) and five rows of C floats.
enum GateRow { kGHi = 0, kGLo = 1, kEG = 2, kRest = 3, kBeta = 4, kGateRows = 5 };

// Sizes, and what every kernel of a call is given.
struct DeltaSizes {
  int64_t T;
  int S, Hk, H, dk, dv;
  const int32_t* offs;
  float scale;
};

constexpr int kDeltaMaxDim = 128;
inline int64_t delta_tiles(int64_t T, int64_t S, int dtype) {
  return (T >> (dtype == DET_BF16 ? DeltaType<uint16_t>::kLogC : DeltaType<float>::kLogC)) + S;
}

// Host: launches of the preparing kernel, and the common checks of the calls.
void delta_prepare(const DeltaSizes& z, int dtype, const void* k, int64_t k_st, int64_t k_sh, const float* g, int64_t g_ld,
                   const void* beta, int64_t beta_ld, float* inverse, float* gates, hipStream_t st);
int delta_check_sizes(const char* what, int dtype, int64_t T, int64_t S, int64_t Hk, int64_t H, int64_t dk, int64_t dv);
// The buffer of a [T, heads, dim] tensor, or an error where its strides are not those
// of whole tokens or of whole heads.
int delta_buf(const char* what, const char* name, const void* p, int64_t T, int64_t heads, int64_t dim, int64_t st, int64_t sh,
              size_t elem, Buf& out);

}  // namespace detgrad
