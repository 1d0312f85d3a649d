// Building blocks of the gated delta rule's kernels: 16 x 16 tiles on the matrix
// cores with operands in one to three bf16 words, and their fragments in memory.
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
// operands with the places 8 g .. 8 g + 7 of the summed index (32 of them), and gives it
// the rows 4 g + r (r = 0..3) of column c of the result. Which token or channel a
// tile's row stands for is free. Row x of tile i is number
//
//   rho(i, x) = 32 (i / 2) + 8 (x / 4) + 4 (i % 2) + x % 4
//
// here, so a lane's results of tiles 2m and 2m + 1 are the eight neighbours 32 m + 8 g ..
// and, as they stand, its places in the next product: a chain of products keeps its
// running operand in registers, and an operand's fragment from memory is 16 bytes of a
// row (of K as it is given, say).
#pragma once

#include "rowops.hpp"
#include "segtiles.hpp"

namespace detgrad {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ constexpr int rho(int tile, int x) {
  return 32 * (tile >> 1) + 8 * (x >> 2) + 4 * (tile & 1) + (x & 3);
}
// and back: the tile and the row in it of a number
__device__ __forceinline__ constexpr int rho_tile(int n) { return 2 * (n >> 5) + ((n >> 2) & 1); }
__device__ __forceinline__ constexpr int rho_row(int n) { return 4 * ((n >> 3) & 3) + (n & 3); }

// f(0), f(1), .. f(N - 1) with constant arguments.
template <int I>
struct Index {
  static constexpr int value = I;
};
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(const F& f) {
  if constexpr (I < N) {
    f(Index<I>{});
    static_for<N, I + 1>(f);
  }
}

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
// acc[t] += A[t] B (SWAP: B A[t]) for the tiles t in [FROM, TO), their terms in turn: one
// after the other would wait for its own result each time.
template <int P, int FROM, int TO, bool SWAP = false, int N, int NA, int NB>
__device__ __forceinline__ void mm_tiles(f32x4 (&acc)[N], const Frag<NA> (&a)[N], const Frag<NB>& b) {
#pragma unroll
  for (int s = P - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB)
#pragma unroll
        for (int t = FROM; t < TO; ++t)
          acc[t] = SWAP ? __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.w[s - i], a[t].w[i], acc[t], 0, 0, 0)
                        : __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t].w[i], b.w[s - i], acc[t], 0, 0, 0);
}

// The words of two values side by side (one conversion instruction for both; taking a word from
// its value with the dot product instruction instead of unpacking it was slower: 572 for 507 us).
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <int NP>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&w)[NP]) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const f32x2 v = {x, y};
    w[p] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    if (p + 1 < NP) {
      x -= bf16_lo(w[p]);
      y -= bf16_hi(w[p]);
    }
  }
}

// The fragment whose places are the rows of two results (or any eight values).
template <int NP>
__device__ __forceinline__ Frag<NP> frag_of(const f32x4& x, const f32x4& y) {
  uint32_t w[4][NP];
  split2<NP>(x[0], x[1], w[0]);
  split2<NP>(x[2], x[3], w[1]);
  split2<NP>(y[0], y[1], w[2]);
  split2<NP>(y[2], y[3], w[3]);
  Frag<NP> f;
#pragma unroll
  for (int p = 0; p < NP; ++p) f.w[p] = __builtin_bit_cast(bf16x8, u32x4{w[0][p], w[1][p], w[2][p], w[3][p]});
  return f;
}

// The value itself, of which the compiler knows nothing: what is computed from it in a
// loop stays there. (Moved out, the addresses of a chunk's loads fill the registers.)
template <typename V>
__device__ __forceinline__ V here(V x) {  // the same for the wave
  asm volatile("" : "+s"(x));
  return x;
}
template <typename V>
__device__ __forceinline__ V here_lane(V x) {
  asm volatile("" : "+v"(x));
  return x;
}

// A value `off` bytes from `base`, the same for the wave: the address is then a scalar
// and one register (pointers of the lanes' own take two and 64-bit sums).
template <typename V>
__device__ __forceinline__ V load_at(const void* base, uint32_t off) {
  V v;
  __builtin_memcpy(&v, static_cast<const char*>(base) + off, sizeof(V));
  return v;
}

// Images: fragments one after the other, each NP words of 64 lanes of 16 bytes.
constexpr int kFragElems = 64 * 8;
// One of them, its first NP words, from LDS.
template <int NP, int STORED>
__device__ __forceinline__ Frag<NP> lds_frag(const char* image, int f) {
  static_assert(NP <= STORED, "more words than the image has");
  Frag<NP> r;
#pragma unroll
  for (int p = 0; p < NP; ++p)
    r.w[p] = *reinterpret_cast<const bf16x8*>(image + (f * STORED + p) * 1024 + (threadIdx.x & 63) * 16);
  return r;
}
template <int NP>
__device__ __forceinline__ void image_put(uint16_t* image, int f, const Frag<NP>& v) {
#pragma unroll
  for (int p = 0; p < NP; ++p) __builtin_memcpy(image + (f * NP + p) * kFragElems + (threadIdx.x & 63) * 8, &v.w[p], 16);
}
// Images of rows as they come from a tensor (fetch_rows): lane 16 g + c of a fragment lies at
// place 16 g + (c ^ 4 g), which keeps the reads of turned_frag on banks of their own.
__device__ __forceinline__ int row_place() {
  const int lane = threadIdx.x & 63;
  return lane ^ (lane >> 4 << 2);
}
template <int NP>
__device__ __forceinline__ Frag<NP> row_frag(const char* image, int f) {
  Frag<NP> r;
#pragma unroll
  for (int p = 0; p < NP; ++p) r.w[p] = *reinterpret_cast<const bf16x8*>(image + (f * NP + p) * 1024 + row_place() * 16);
  return r;
}
// From an image of rows t and places d (KD fragments per tile), the fragment of rows d, tile j,
// and places t, 32 kt + 8 g ..: the hardware reads 16 columns of four rows, turned, for the lanes
// of a group; lane p of it gives the address of four columns, 4 (p % 4) .., of row p / 4.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ s16x4 lds_turned4(const char* p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
}
template <int NP>
__device__ __forceinline__ Frag<NP> turned_frag(const char* image, int j, int frag0, int frag1) {  // (of the two row tiles)
  const int lane = threadIdx.x & 63, p = lane & 15, x = 4 * (lane >> 4) + (p >> 2), g = p & 3;
  const char* at = image + (16 * g + (x ^ (4 * g))) * 16 + 8 * (j & 1);
  Frag<NP> r;
#pragma unroll
  for (int w = 0; w < NP; ++w) {
    const s16x4 a = lds_turned4(at + (frag0 * NP + w) * 1024), b = lds_turned4(at + (frag1 * NP + w) * 1024);
    r.w[w] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  return r;
}
template <int KD, int NP>
__device__ __forceinline__ Frag<NP> turned_frag(const char* image, int j, int kt) {
  return turned_frag<NP>(image, j, 2 * kt * KD + (j >> 1), (2 * kt + 1) * KD + (j >> 1));
}
// The first NP words to LDS.
template <int NP, int N>
__device__ __forceinline__ void lds_put(char* image, int f, const Frag<N>& v) {
#pragma unroll
  for (int p = 0; p < NP; ++p) *reinterpret_cast<bf16x8*>(image + (f * NP + p) * 1024 + (threadIdx.x & 63) * 16) = v.w[p];
}
// Square images [C][C] of lower (rows i, places j <= i) or upper (rows j, places i >= j)
// triangles leave out the fragments that hold nothing else: their numbers.
__device__ __forceinline__ constexpr int lower_frag(int i, int kt) { return (i >> 1) * ((i >> 1) + 1) + (i & 1) * ((i >> 1) + 1) + kt; }
template <int KC>
__device__ __forceinline__ constexpr int upper_frag(int j, int kt) {
  return 2 * ((j >> 1) * KC - (j >> 1) * ((j >> 1) - 1) / 2) + (j & 1) * (KC - (j >> 1)) + kt - (j >> 1);
}

// At the end of one of two ways to load the same: keeps the compiler from joining their
// loads into one sequence with the addresses of either in registers.
__device__ __forceinline__ void own_way() { asm volatile("; its own way" ::: "memory"); }

// Four consecutive elements at .. at + 3 of a row of n, those behind it zero, loaded
// without a branch (loads under one would be waited for one by one): whole rows (n a
// multiple of four, the same for all) in one access, others element by element.
template <typename T>
__device__ __forceinline__ f32x4 load4(const T* row, int at, int n, bool whole) {
  T v[4];
  if (whole) {
    __builtin_memcpy(v, row + (at < n ? at : 0), 4 * sizeof(T));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = row[at + j < n ? at + j : n - 1];
    own_way();
  }
  f32x4 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = at + j < n ? to_f32(v[j]) : 0.0f;
  return r;
}
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
  uint32_t a[1], b[1];
  split2<1>(v[0], v[1], a);
  split2<1>(v[2], v[3], b);
  if (n >= 4) {
    const uint64_t w = a[0] | static_cast<uint64_t>(b[0]) << 32;
    __builtin_memcpy(p, &w, 8);
  } else {
    if (n > 0) p[0] = static_cast<uint16_t>(a[0]);
    if (n > 1) p[1] = static_cast<uint16_t>(a[0] >> 16);
    if (n > 2) p[2] = static_cast<uint16_t>(b[0]);
  }
}
// Results with rows v0 + 4 g + r and columns t = rho(i, c) < n: x[i][r] to place v0 + 4 g + r of row t.
template <int RT, typename T>
__device__ __forceinline__ void store_rows(const f32x4 (&x)[RT], T* rows, int64_t st, int v0, int dv, int n) {
  const int lane = here_lane(threadIdx.x) & 63, c = lane & 15, v = v0 + 4 * (lane >> 4);
  T* to = rows + rho(0, c) * st + v;
  if (n == 16 * RT && v0 + 16 <= dv) {  // (the same for all)
#pragma unroll
    for (int i = 0; i < RT; ++i) store4(to + rho(i, 0) * st, 4, x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < RT; ++i)
      if (rho(i, c) < n) store4(to + rho(i, 0) * st, dv - v, x[i]);
  }
}

// Memory to LDS past the registers: N groups of 64 lanes of 16 bytes; lane l brings those at
// base + off[j] + 1024 j to `lds` + 1024 j + 16 l (the instruction's offset counts on both
// sides; base and lds the same for the wave). In assembly, since the compiler makes every
// read of LDS wait for all such loads, those of a buffer that is only read later
// too; the wait is fetch_done() and a barrier. It counts only its own loads, of which
// there are fewer than the hardware counts, so its waits are never too short.
typedef __attribute__((address_space(3))) void lds_void;
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)p));
}
#define DET_FETCH_HEAD "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\t"
#define DET_FETCH_TAIL "s_mov_b32 m0, %0"
template <int N>
__device__ __forceinline__ void fetch_group(uint32_t lds, const void* base, const uint32_t (&off)[N]) {
  static_assert(N >= 1 && N <= 4, "offsets up to 4095 bytes");
  uint32_t m0;
  lds = __builtin_amdgcn_readfirstlane(lds);
  if constexpr (N == 1)
    asm volatile(DET_FETCH_HEAD DET_FETCH_TAIL : "=&s"(m0) : "s"(lds), "v"(off[0]), "s"(base) : "memory");
  if constexpr (N == 2)
    asm volatile(DET_FETCH_HEAD "global_load_lds_dwordx4 %4, %3 offset:1024\n\t" DET_FETCH_TAIL
                 : "=&s"(m0) : "s"(lds), "v"(off[0]), "s"(base), "v"(off[1]) : "memory");
  if constexpr (N == 3)
    asm volatile(DET_FETCH_HEAD "global_load_lds_dwordx4 %4, %3 offset:1024\n\tglobal_load_lds_dwordx4 %5, %3 offset:2*1024\n\t"
                 DET_FETCH_TAIL : "=&s"(m0) : "s"(lds), "v"(off[0]), "s"(base), "v"(off[1]), "v"(off[2]) : "memory");
  if constexpr (N == 4)
    asm volatile(DET_FETCH_HEAD "global_load_lds_dwordx4 %4, %3 offset:1024\n\tglobal_load_lds_dwordx4 %5, %3 offset:2*1024\n\t"
                 "global_load_lds_dwordx4 %6, %3 offset:3*1024\n\t" DET_FETCH_TAIL
                 : "=&s"(m0) : "s"(lds), "v"(off[0]), "s"(base), "v"(off[1]), "v"(off[2]), "v"(off[3]) : "memory");
}
#undef DET_FETCH_HEAD
#undef DET_FETCH_TAIL
__device__ __forceinline__ void fetch_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// All but the last N of this wave.
template <int N>
__device__ __forceinline__ void fetch_done_but() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N < 63 ? N : 63) : "memory");
}
// What this wave has read of LDS is in its registers (a fetch may write there).
__device__ __forceinline__ void lds_read() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// N consecutive fragments of an image, four at a time, shared out among NW waves from wave FIRST on.
template <int N, int NW, int FIRST = 0>
__device__ __forceinline__ void fetch_image(uint32_t lds, const uint16_t* image, int wave) {
  const uint32_t l = (threadIdx.x & 63) * 16;
  wave = here(wave);
  static_for<(N + 3) / 4>([&](auto group) {
    constexpr int f = 4 * group.value, n = N - f < 4 ? N - f : 4;
    uint32_t off[n];
#pragma unroll
    for (int j = 0; j < n; ++j) off[j] = l;
    if (NW == 1 || wave == (group.value + FIRST) % NW) fetch_group<n>(lds + f * 1024, image + f * kFragElems, off);
  });
}

// Writes to LDS of this wave's lanes are seen by its other lanes after this (the
// wave's LDS accesses run in order; the compiler must not reorder them).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Results with rows v0 + 4 g + r and columns rho(i, c) as a part of a float32 image with rows t and
// places v (kv fragments of 32 per row tile), zeros from place dv on, nothing behind the image's. A fragment is the first
// four of its 64 lanes' eight places, then the others, so that it is stored and loaded in whole lines.
constexpr int kFragFloats = 64 * 8;
template <int RT>
__device__ __forceinline__ void put_image(const f32x4 (&x)[RT], float* image, int v0, int dv, int kv) {
  const int lane = threadIdx.x & 63, c = lane & 15, v = v0 + 4 * (lane >> 4);
  if (v0 >= 32 * kv) return;
  float* to = image + (v >> 5) * kFragFloats + ((v >> 2) & 1) * 256 + (16 * ((v >> 3) & 3) + c) * 4;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    f32x4 y;
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] = v + r < dv ? x[i][r] : 0.0f;
    *reinterpret_cast<f32x4*>(to + i * kv * kFragFloats) = y;
  }
}

__device__ __forceinline__ f32x4 gate4(const float* gate, int C, int row, int at) {
  return *reinterpret_cast<const f32x4*>(gate + row * C + at);
}

// A result tile (rows 4 g + r, column c) in 1024 bytes of LDS, and back with rows and columns changed;
// lane 16 g + c at place 16 g + (c ^ g), so that the latter reads every bank once.
__device__ __forceinline__ f32x4* lds_tile(char* at) {
  const int lane = threadIdx.x & 63;
  return reinterpret_cast<f32x4*>(at) + (lane ^ (lane >> 4));
}
__device__ __forceinline__ f32x4 lds_turned(const char* at) {
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const char* p = at + (16 * (c >> 2) + 4 * g) * 16 + (c & 3) * 4;
  f32x4 v;
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = *reinterpret_cast<const float*>(p + 16 * (r ^ (c >> 2)));
  return v;
}
// The tiles of a result with rows and columns changed, in 2048 bytes of this wave.
template <int RT>
__device__ __forceinline__ void turn_tiles(f32x4 (&y)[RT], const f32x4 (&x)[RT], char* scratch) {
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    char* tile = scratch + (i & 1) * 1024;
    *lds_tile(tile) = x[i];
    wave_fence();
    y[i] = lds_turned(tile);
    wave_fence();
  }
}

// A [T, heads, dim] tensor with unit innermost stride.
template <typename T>
struct Heads {
  T* p;
  int64_t st, sh;
  __device__ __forceinline__ T* row(int64_t t, int h) const { return p + t * st + h * sh; }
};

// The elements of a chunk's rows t0 + rho(i, 4 g + r) in one column, `col` elements from
// `rows` on (row t0 of the head): unconditional loads, the row `last` again behind it.
template <int RT, typename T>
__device__ __forceinline__ void load_column(T (&v)[RT][4], const T* rows, int64_t st, int col, int last) {
  const int g = (here_lane(threadIdx.x) & 63) >> 4;
  st = here(st);
  if (last == 16 * RT - 1 && st < (1 << 24)) {  // (the same for all) whole chunks: the rows' distances are uniform
    const uint32_t off = (8u * g * static_cast<uint32_t>(st) + col) * sizeof(T);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[i][r] = load_at<T>(rows + rho(i, r) * st, off);
  } else {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = rho(i, 4 * g + r);
        v[i][r] = rows[(t < last ? t : last) * st + col];
      }
    own_way();
  }
}
// The elements d = rho(i, 4 g + r) < dk (others: the first row's) of column col of a [dk, dv] state.
template <int DT>
__device__ __forceinline__ void load_state(float (&v)[DT][4], const float* state, int dk, int dv, int col) {
  const int g = (here_lane(threadIdx.x) & 63) >> 4;
  dv = here(dv);
  const uint32_t off = static_cast<uint32_t>(8 * g * dv + col) * 4u;
  if (dk == 16 * DT) {
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[i][r] = load_at<float>(state + rho(i, r) * dv, off);
  } else {
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = rho(i, 4 * g + r);
        v[i][r] = load_at<float>(state, static_cast<uint32_t>((d < dk ? d : 0) * dv + col) * 4u);
      }
    own_way();
  }
}
template <int DT>
__device__ __forceinline__ void store_state(const f32x4 (&v)[DT], float* state, int dk, int dv, int col) {
  const int g = (here_lane(threadIdx.x) & 63) >> 4;
  dv = here(dv);
  if (dk == 16 * DT) {
    if (col < dv)
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *reinterpret_cast<float*>(reinterpret_cast<char*>(state + rho(i, r) * dv) + static_cast<uint32_t>(8 * g * dv + col) * 4u) = v[i][r];
  } else {
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = rho(i, 4 * g + r);
        if (col < dv && d < dk) state[d * dv + col] = v[i][r];
      }
  }
}

// The same for a state between kernels: [dv / 16][dk][16], of which a wave's columns are one block, so that
// it is stored in whole lines; turned in 2048 bytes of LDS (32 stores of 4 bytes took most of a chunk).
template <int DT>
__device__ __forceinline__ void store_block(const f32x4 (&v)[DT], float* block, int dk, char* scratch) {
  const int lane = here_lane(threadIdx.x) & 63, c = lane & 15;
#pragma unroll
  for (int i = 0; i < DT; ++i) {
    char* tile = scratch + (i & 1) * 1024;
    *lds_tile(tile) = v[i];
    wave_fence();
    const f32x4 w = lds_turned(tile);
    wave_fence();
    if (rho(i, c) < dk) *reinterpret_cast<f32x4*>(block + rho(i, c) * 16 + 4 * (lane >> 4)) = w;
  }
}

// The rows of a [T, heads, dim] operand in bf16 words: a bf16 tensor itself where its
// rows start on 16-byte borders and dim is the kernels' own, else a copy [T, heads, words, dim]
// padded with zeros.
struct Rows {
  const uint16_t* p;
  int64_t st, sh;
  int words_at;  // from word to word
  // the rows from token t of a head on; the places 32 ks + 8 g .. of row t + `row` of them (st < 2^24: see as_it_is)
  __device__ __forceinline__ const uint16_t* from(int64_t t, int h) const { return p + t * st + h * sh; }
  __device__ __forceinline__ uint32_t lane_off(int row) const {
    return (static_cast<uint32_t>(row) * static_cast<uint32_t>(st) + 8u * ((threadIdx.x & 63) >> 4)) * 2u;
  }
  template <int NP>
  __device__ __forceinline__ Frag<NP> frag(const uint16_t* rows, uint32_t off, int ks) const {
    Frag<NP> f;
#pragma unroll
    for (int w = 0; w < NP; ++w) f.w[w] = load_at<bf16x8>(rows + w * words_at + 32 * ks, off);
    return f;
  }
};
// The fragments of a chunk's rows t0 + rho(i, c) (the last one again behind it) as an image
// in LDS, tile by tile, KD places of 32 each, NP words; shared out among NW waves. The rows'
// strides are below 2^24 elements (as_it_is), so that a chunk spans less than 2^32 bytes.
template <int RT, int KD, int NP, int NW, int FIRST = 0>
__device__ __forceinline__ void fetch_rows(uint32_t lds, const Rows& x, int64_t t0, int last, int h, int wave) {
  constexpr int kTile = KD * NP, kGroups = (kTile + 3) / 4;
  const int c = here_lane(row_place()) & 15;
  wave = here(wave);
  const uint16_t* base = x.from(t0, h) - 2048;  // (the offsets below would be negative)
  static_for<RT * kGroups>([&](auto group) {
    constexpr int i = group.value / kGroups, f = 4 * (group.value % kGroups), n = kTile - f < 4 ? kTile - f : 4;
    if (NW == 1 || wave == (group.value + FIRST) % NW) {
      const int t = rho(i, c);
      const uint32_t row = x.lane_off(t < last ? t : last) + 4096u;
      uint32_t off[n];
#pragma unroll
      for (int j = 0; j < n; ++j)
        off[j] = row + 64u * ((f + j) / NP) - 1024u * j + (NP == 1 ? 0u : (f + j) % NP * 64u * KD);  // words: KD * 32 apart
      fetch_group<n>(lds + (i * kTile + f) * 1024, base, off);
    }
  });
}

// 16 columns from v0 on of a chunk's rows (RT tiles) in LDS, 2048 bytes of [row][column], for this
// wave: where `whole_columns`, the rows' strides and starts being whole 16 bytes.
template <typename T>
__device__ __forceinline__ bool whole_columns(const Heads<const T>& x, int v0, int dv) {
  return v0 + 16 <= dv && x.st < (1 << 24) && ((reinterpret_cast<uintptr_t>(x.p) | x.st * sizeof(T) | x.sh * sizeof(T)) & 15) == 0;
}
template <int RT, typename T>
__device__ __forceinline__ void fetch_columns(uint32_t lds, const Heads<const T>& x, int64_t t0, int h, int v0, int last) {
  constexpr int kLanes = sizeof(T);  // of a row
  static_assert(16 * RT * 16 * sizeof(T) == 2048, "two loads");
  const int lane = here_lane(threadIdx.x) & 63;
  const char* base = reinterpret_cast<const char*>(x.row(t0, h) + v0) - 4096;
  uint32_t off[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = j * (64 / kLanes) + lane / kLanes;
    off[j] = static_cast<uint32_t>(t < last ? t : last) * static_cast<uint32_t>(x.st * sizeof(T)) + lane % kLanes * 16 + 4096 - 1024 * j;
  }
  fetch_group<2>(lds, base, off);
}
// The elements of rows rho(i, 4 g + r), column v0 + c, of that.
template <int RT>
__device__ __forceinline__ void take_columns(f32x4 (&v)[RT], const char* lds, const float*) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) v[i][r] = *reinterpret_cast<const float*>(lds + rho(i, r) * 64 + (lane >> 4) * 8 * 64 + (lane & 15) * 4);
}
template <int RT>
__device__ __forceinline__ void take_columns(f32x4 (&v)[RT], const char* lds, const uint16_t*) {
  const int lane = threadIdx.x & 63, p = lane & 15;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const s16x4 w = lds_turned4(lds + (rho(i, 0) + 8 * (lane >> 4) + (p >> 2)) * 32 + (p & 3) * 8);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[i][r] = to_f32(static_cast<uint16_t>(w[r]));
  }
}

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

// S = el S + X^T y, from X's rows in LDS (`image`) and the fragments of y, and S's own
// fragments: in two halves, so that the words of one are made under the products of the other.
template <int NP, int KC, int DT, int N>
__device__ __forceinline__ void next_state(f32x4 (&S)[DT], Frag<N> (&f)[DT / 2], const char* image, const Frag<N> (&y)[KC], float el) {
#pragma unroll
  for (int i = 0; i < DT; ++i) S[i] *= el;
  static_for<2>([&](auto half) {
    constexpr int from = half.value * DT / 2, to = from + DT / 2;
#pragma unroll
    for (int kt = 0; kt < KC; ++kt) {
      Frag<NP> ft[DT];
#pragma unroll
      for (int i = from; i < to; ++i) ft[i] = turned_frag<DT / 2, NP>(image, i, kt);
      mm_tiles<N, from, to>(S, ft, y[kt]);
    }
    if constexpr (half.value == 0) {
      __builtin_amdgcn_sched_barrier(0);
    } else {
#pragma unroll
      for (int i = 0; i < from; i += 2) f[i / 2] = frag_of<N>(S[i], S[i + 1]);
      // an instruction of the matrix cores, then four others, in turn
      static_for<KC * DT / 2 * N * (N + 1) / 2>([](auto) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
      });
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = from; i < to; i += 2) f[i / 2] = frag_of<N>(S[i], S[i + 1]);
    }
  });
}

// Tokens per chunk, words of an input. float32 takes half the chunk: its operands have three words.
template <typename T>
struct DeltaType;
template <>
struct DeltaType<uint16_t> {
  static constexpr int kLogC = 6, kIn = 1;
};
template <>
struct DeltaType<float> {
  static constexpr int kLogC = 5, kIn = 3;
};
// Words of everything else, states and what is only ever rounded to bf16 alike. (o of a bf16 call in two words, 16 bits:
// 0.35 % of its values were another bf16 value than the rounded exact one, in three 0.01 to 0.03 % as from float32;
// 32768 tokens 1254 and 1293 us. The gradients: see delta_bwd.hip.)
constexpr int kStateWords = 3;

// exp(hi + lo) of a difference of two-word sums
__device__ __forceinline__ float decay(float hi_i, float lo_i, float hi_j, float lo_j) {
  return exp_e((hi_i - hi_j) + (lo_i - lo_j));
}

// Rows of C floats that the preparing kernel leaves per (chunk, value head): the running
// of g in two words, exp(G) and beta (0 behind the sequence's end), exp(G_C - G),
// exp(G_C) in every place, and the products exp(G_C - G) beta and -exp(G) beta.
enum GateRow { kGHi = 0, kGLo = 1, kEG = 2, kRest = 3, kBeta = 4, kEnd = 5, kRestBeta = 6, kEGBeta = 7, kGateRows = 8 };

// What it leaves per (chunk, value head), in fragments of 1024 bytes: the inverse, those rows, P.
template <typename T, bool BWD>
struct Unit {
  static constexpr int C = 1 << DeltaType<T>::kLogC, KC = C / 32, kFrags = KC * (KC + 1);
  static constexpr int nInv = kFrags * kStateWords, nGate = (kGateRows * C * 4 + 1023) / 1024, nP = kFrags * kStateWords;
  static constexpr int oGate = nInv, oP = nInv + nGate, nAll = oP + nP, kElems = nAll * kFragElems;
};

// Sizes, and what every kernel of a call is given.
struct DeltaSizes {
  int64_t T;
  int S, Hk, H, dk, dv;
  const int32_t* offs;
  float scale;
};

constexpr int kDeltaMaxDim = 128;
inline int delta_chunk(int dtype) { return 1 << (dtype == DET_BF16 ? DeltaType<uint16_t>::kLogC : DeltaType<float>::kLogC); }
inline int delta_words(int dtype) { return dtype == DET_BF16 ? DeltaType<uint16_t>::kIn : DeltaType<float>::kIn; }
inline int64_t delta_tiles(int64_t T, int64_t S, int dtype) { return T / delta_chunk(dtype) + S; }
inline int delta_pad(int64_t d) { return d <= 64 ? 64 : 128; }

// The workgroups of the chains of states: eight waves for all columns of a head, which share its
// fragments, or a team of three waves for 16 columns. A team's chunk takes 2.2 us, the eight waves'
// 5.9 to 6.5 us, but there are eight times as many teams for the compute units. Whole calls of 32 heads with sequences of
// equal length, teams and eight waves, us:
//   8192 tokens, 128 x 128, bf16, forward: one sequence 372 and 927, two 352 and 505, three 368 and 380, eight 373 and 200;
//     with the backward's states 510 and 1088, 512 and 611, 533 and 473, 531 and 263; backward, two and three: 877 and
//     988, 886 and 838
//   4096 tokens, 128 x 128, float32, forward: two 380 and 509, three 387 and 392, eight 403 and 257
//   64 x 64 halves the teams, which are better up to about 160 chains there: forward of 8192 tokens in bf16, three 201 and
//     281, four 164 and 221, five 197 and 201, eight 170 and 151
// The bound is that of 128 columns for all. The lengths are on the device: sequences without tokens count too.
inline bool delta_teams(const DeltaSizes& z) { return static_cast<int64_t>(z.S) * z.H <= 80; }

// What a forward leaves for the backward per (chunk, value head), in floats: N as an image of rows t and
// places v, then the state in front of the chunk in blocks of 16 columns.
inline int64_t delta_image_floats(int64_t dv, int dtype) { return delta_chunk(dtype) * delta_pad(dv); }
inline int64_t delta_block_floats(int64_t dk, int64_t dv) { return dk * static_cast<int64_t>(align_up(static_cast<size_t>(dv), 16)); }
inline int64_t delta_saved_floats(int64_t dk, int64_t dv, int dtype) { return delta_image_floats(dv, dtype) + delta_block_floats(dk, dv); }

// Where the parts of a workspace lie. units: a Unit each; dy: the backward's images as N's.
struct DeltaLayout {
  size_t units, k_rows, q_rows, o_rows, ds, dy, all;
};
DeltaLayout delta_layout(const DeltaSizes& z, int dtype, bool bwd);

// Host: the kernels that every call begins with, and the common checks of the calls.
struct DeltaPrepared {
  Rows k, q, d_o;
};
DeltaPrepared delta_prepare(const DeltaSizes& z, int dtype, bool bwd, const void* q, int64_t q_st, int64_t q_sh, const void* k,
                            int64_t k_st, int64_t k_sh, const void* d_o, int64_t do_st, int64_t do_sh, const float* g,
                            int64_t g_ld, const void* beta, int64_t beta_ld, char* ws, const DeltaLayout& l, hipStream_t st);
int delta_check_sizes(const char* what, int dtype, int64_t T, int64_t S, int64_t Hk, int64_t H, int64_t dk, int64_t dv);
// The buffer of a [T, heads, dim] tensor, or an error where its strides are not those
// of whole tokens or of whole heads.
int delta_buf(const char* what, const char* name, const void* p, int64_t T, int64_t heads, int64_t dim, int64_t st, int64_t sh,
              size_t elem, Buf& out);

}  // namespace detgrad
