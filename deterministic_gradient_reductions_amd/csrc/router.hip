// det_router_balance / det_router_balance_bwd: the router's load-balancing loss
// with its per-expert counts and score sums, and the gradient of its logits.
//
//   p[t]         = softmax(z[t]), or sigmoid(z[t]) / sum sigmoid(z[t]) (the softmax of log sigmoid(z))
//   counts[s][e] = slots (t, k) of segment s with ids[t][k] == e
//   P[s][e]      = sum of p[t][e] over the tokens of segment s
//   loss[s]      = coeff E / (K N_s^2) sum_e counts[s][e] P[s][e]
//   dz[t][e]     = dloss[s] coeff E / (K N_s^2) p_e (c_e - sum_j p_j c_j)   [(1 - sigmoid(z_e)) for the sigmoid score]
//
// Layout: a row of E logits sits in LPR lanes of NI times eight consecutive
// columns, 64 / LPR rows per wave and step, so a row's maximum and sums are a few
// lane exchanges (for two times eight columns per lane half as many as for eight)
// and every lane keeps the running P of its own columns in registers.
//
// Order of P (no atomics): a tile of rows of one segment belongs to one
// workgroup; lane group g of wave w adds its rows of the tile in ascending
// order, the lane groups of a wave meet in an adjacent tree, the waves left to
// right, and the tile's sum is one float32 slot. The fold adds a segment's
// slots in float64, in tile order per strip and the strips in order. Counts are
// whole numbers, so their LDS atomics have one result.
//
// Bytes: the logits once per direction, dz once. Measured at 65536 x 256 bf16
// with sigmoid scores, 16 segments: tiles 13.5 us (33.5 MB read; the vector units
// busy for 6.9), fold 5.5, backward 15.9 (67 MB; busy for 9.2): at this size the
// chain offsets -> rows -> sums -> slots still costs as much as the bytes (13 us in
// all at the rate of a copy), and small calls are bound by their launches.
#include "rowops.hpp"
#include "segtiles.hpp"

namespace detgrad {
namespace {

constexpr int kFwdThreads = 512, kDirectThreads = 1024, kBwdThreads = 256, kFoldThreads = 1024;

// Offsets of up to this many groups of 64 segments are fetched together where
// the offsets are scanned.
constexpr int kScanBatch = 8;

// Rows of a lane group whose loads are in flight together (half as many where a
// lane holds sixteen columns).
constexpr int fwd_ahead(int ni) { return 2 / ni; }
constexpr int bwd_ahead(int ni) { return 2 / ni; }

// exp(x) for x <= 0 as 2^(x log2 e): within (|x| + 2) units in the last place,
// which is below 2^-24 of the row's largest score (its own error is |x| e^x).
__device__ __forceinline__ float exp_nonpos(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// The maximum taken out of a row's exponents; 0 for a row of nothing but -inf,
// whose scores are then all exp(-inf) = 0 (and a NaN stays one).
template <int LPR, int NI>
__device__ __forceinline__ float row_max(const float (&z)[NI][8]) {
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, z[i][j]);
  m = lanes_max<LPR>(m);
  return m == -__builtin_inff() ? 0.0f : m;
}
template <int LPR, int NI>
__device__ __forceinline__ float row_sum(const float (&e)[NI][8]) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i)
    s += ((e[i][0] + e[i][1]) + (e[i][2] + e[i][3])) + ((e[i][4] + e[i][5]) + (e[i][6] + e[i][7]));
  return lanes_sum<LPR>(s);
}

// A row's unnormalised scores e (0 in columns of -inf) and 1 / their sum (0 for
// a row without any); q = sigmoid(-z) for the gradient.
// softmax: e = exp(z - max z). sigmoid: e = 1 / (1 + t), q = t e with t =
// exp(-z), which needs no maximum; a row whose scores sum to less than kLowSum
// (every logit below -14) takes e = exp(min(z, 0) - max min(z, 0)) / (1 + exp(-|z|))
// instead, the same scores times a common factor. In any other row the largest
// score is at least 2^-30, so what the first form drops (scores below 2^-126) is
// below 2^-96 of it. The choice is the row's own, not its wave's: a row has the
// same bits whatever rows it is computed beside.
constexpr float kLowSum = 0x1p-20f;
template <int LPR, int NI, bool SIGMOID, bool GRAD>
__device__ __forceinline__ float row_scores(const float (&z)[NI][8], float (&e)[NI][8], float (&q)[NI][8]) {
  float s;
  if constexpr (SIGMOID) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = __builtin_amdgcn_exp2f(z[i][j] * -kLog2e);
        e[i][j] = __builtin_amdgcn_rcpf(1.0f + t);
        if (GRAD) q[i][j] = fminf(t, 0x1p126f) * e[i][j];  // (t = inf: e = 0, and q does not matter)
      }
    s = row_sum<LPR, NI>(e);
    if (__ballot(s < kLowSum) != 0) {
      keep_branch();
      const float m = fminf(row_max<LPR, NI>(z), 0.0f);
      if (s < kLowSum) {  // (the same for the row's lanes)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float t = exp_nonpos(-fabsf(z[i][j])), r = __builtin_amdgcn_rcpf(1.0f + t);
            e[i][j] = exp_nonpos(fminf(z[i][j], 0.0f) - m) * r;
            if (GRAD) q[i][j] = z[i][j] < 0.0f ? r : t * r;
          }
      }
      s = row_sum<LPR, NI>(e);
    }
  } else {
    const float m = row_max<LPR, NI>(z);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) e[i][j] = exp_nonpos(z[i][j] - m);
    s = row_sum<LPR, NI>(e);
  }
  return s == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(s);
}

// The next rows of a wave's lane groups, `AHEAD` per group, W RPW apart, loaded
// together; those past r1 repeat row r0 (and are not used).
template <typename T, int LPR, int NI, int AHEAD>
__device__ __forceinline__ void load_rows(const T* __restrict__ z, int64_t ld, uint32_t r, uint32_t step, uint32_t r0,
                                          uint32_t r1, const Cols<LPR == 1> (&c)[NI], float (&v)[AHEAD][NI][8]) {
  Raw8<T> raw[AHEAD][NI];
#pragma unroll
  for (int a = 0; a < AHEAD; ++a) {
    const uint32_t row = r + a * step < r1 ? r + a * step : r0;
#pragma unroll
    for (int i = 0; i < NI; ++i) load_cols(raw[a][i], z + static_cast<int64_t>(row) * ld, c[i]);
  }
#pragma unroll
  for (int a = 0; a < AHEAD; ++a)
#pragma unroll
    for (int i = 0; i < NI; ++i) raw[a][i].get(v[a][i]);
  if (!c[0].all) {
    keep_branch();
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[a][i][j] = c[i].own(j) ? v[a][i][j] : -__builtin_inff();
  }
}

// P of the rows [r0, r1) into part[0][0..E) and their counts into hist (both
// LDS), by the whole workgroup; ends with the barrier that makes them visible.
// Lane group g of wave w takes rows r0 + w RPW + g, then every W RPW-th row.
template <typename T, int LPR, int NI, bool SIGMOID, int THREADS>
__device__ __forceinline__ void sum_rows(const T* __restrict__ z, int64_t ld, int E, const int32_t* __restrict__ ids,
                                         int64_t ids_ld, int K, uint32_t r0, uint32_t r1,
                                         float (&part)[THREADS / 64][8 * LPR * NI], int32_t (&hist)[8 * LPR * NI]) {
  constexpr int RPW = 64 / LPR, W = THREADS / 64, COLS = 8 * LPR * NI, kAhead = fwd_ahead(NI);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane / LPR, l = lane % LPR;
  for (int i = threadIdx.x; i < COLS; i += THREADS) hist[i] = 0;
  __syncthreads();
  Cols<LPR == 1> c[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) c[i].set((i * LPR + l) * 8, E, COLS);
  // the ids of slots i, i + THREADS, ... (past the last: the first again, and not counted); the first round's are
  // fetched ahead of the rows
  const uint32_t slots = (r1 - r0) * static_cast<uint32_t>(K);  // < 2^31 (checked by the host)
  int32_t id[4];
  const auto fetch_ids = [&](uint32_t i) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t at = i + k * THREADS < slots ? i + k * THREADS : i, r = at / static_cast<uint32_t>(K);
      id[k] = ids[static_cast<int64_t>(r0 + r) * ids_ld + (at - r * K)];
    }
  };
  if (threadIdx.x < slots) fetch_ids(threadIdx.x);
  float acc[NI][8] = {};
  for (uint32_t r = r0 + wave * RPW; r < r1; r += kAhead * W * RPW) {
    float v[kAhead][NI][8];
    load_rows<T, LPR, NI, kAhead>(z, ld, r + sub, W * RPW, r0, r1, c, v);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      float e[NI][8], q[NI][8];
      const float inv = row_scores<LPR, NI, SIGMOID, false>(v[a], e, q);
      if (r + sub + a * W * RPW < r1) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[i][j] = __builtin_fmaf(e[i][j], inv, acc[i][j]);
      }
    }
  }
  for (uint32_t i = threadIdx.x; i < slots; i += 4 * THREADS) {
    if (i >= 4 * THREADS) fetch_ids(i);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * THREADS < slots && id[k] >= 0 && id[k] < E) atomicAdd(&hist[id[k]], 1);
  }
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int d = LPR; d < 64; d <<= 1) acc[i][j] += __shfl_xor(acc[i][j], d);
      if (sub == 0 && c[i].own(j)) part[wave][c[i].base + j] = acc[i][j];
    }
  __syncthreads();
  for (int c = threadIdx.x; c < E; c += THREADS) {
    float s = part[0][c];
#pragma unroll
    for (int w = 1; w < W; ++w) s += part[w][c];
    part[0][c] = s;  // column c belongs to this thread alone
  }
}

template <typename T, int LPR, int NI, bool SIGMOID>
__global__ __launch_bounds__(kFwdThreads) void router_tile_kernel(const T* __restrict__ z, int64_t ld, uint32_t rows,
                                                                  int E, const int32_t* __restrict__ ids,
                                                                  int64_t ids_ld, int K,
                                                                  const int32_t* __restrict__ offs, int S, int log_bt,
                                                                  float* __restrict__ slot_p,
                                                                  int32_t* __restrict__ slot_c,
                                                                  int32_t* __restrict__ table) {
  __shared__ float part[kFwdThreads / 64][8 * LPR * NI];
  __shared__ int32_t hist[8 * LPR * NI];
  if (blockIdx.x == 0 && threadIdx.x < 64) write_tile_table(offs, S, rows, log_bt, table);
  int seg;
  uint32_t r0, r1, s0, s1;
  if (!segment_tile<kScanBatch>(offs, S, rows, log_bt, blockIdx.x, seg, r0, r1, s0, s1)) return;  // the grid covers the worst case
  sum_rows<T, LPR, NI, SIGMOID, kFwdThreads>(z, ld, E, ids, ids_ld, K, r0, r1, part, hist);
  for (int c = threadIdx.x; c < E; c += kFwdThreads) {
    slot_p[static_cast<int64_t>(blockIdx.x) * E + c] = part[0][c];
    slot_c[static_cast<int64_t>(blockIdx.x) * E + c] = hist[c];
  }
}

// [b_s, b_{s+1}): the running maximum of the clamped offsets, by every wave.
__device__ __forceinline__ void segment_bounds(const int32_t* __restrict__ offs, int s, uint32_t rows, uint32_t& b0,
                                               uint32_t& b1) {
  const uint32_t last = clamp_off(offs[s + 1], rows);
  uint32_t b = 0;
  for (int i = 0; i <= s; i += 64 * kScanBatch) {
    uint32_t v[kScanBatch] = {};
#pragma unroll
    for (int k = 0; k < kScanBatch; ++k) {
      if (k > 0 && i + 64 * k > s) break;  // (the same for every lane)
      const int at = i + 64 * k + static_cast<int>(threadIdx.x & 63);
      v[k] = clamp_off(offs[at <= s ? at : s], rows);
    }
#pragma unroll
    for (int k = 0; k < kScanBatch; ++k) b = umax(b, v[k]);
  }
  b0 = lane_value(scan_max(b), 63);
  b1 = umax(b0, last);
}

__device__ __forceinline__ double balance_scale(double coeff, int E, int K, uint32_t n) {
  return n == 0 ? 0.0 : coeff * E / (static_cast<double>(K) * n * n);
}

// A segment's outputs from its sums, by the first E threads' columns: returns
// nothing; loss = scale sum_e counts P in float64, adjacent tree per wave, waves
// left to right.
template <int THREADS>
__device__ __forceinline__ void write_loss(double term, double scale, float* __restrict__ loss,
                                           double (&sl)[THREADS / 64]) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) term += __shfl_xor(term, d);
  if ((threadIdx.x & 63) == 0) sl[threadIdx.x >> 6] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    double tot = sl[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) tot += sl[w];
    *loss = static_cast<float>(scale * tot);
  }
}

// The whole forward of a small call in one launch: workgroup s sums all tokens
// of segment s.
template <typename T, int LPR, int NI, bool SIGMOID>
__global__ __launch_bounds__(kDirectThreads) void router_direct_kernel(const T* __restrict__ z, int64_t ld,
                                                                       uint32_t rows, int E,
                                                                       const int32_t* __restrict__ ids,
                                                                       int64_t ids_ld, int K,
                                                                       const int32_t* __restrict__ offs, double coeff,
                                                                       float* __restrict__ psum,
                                                                       int32_t* __restrict__ counts,
                                                                       float* __restrict__ loss) {
  __shared__ float part[kDirectThreads / 64][8 * LPR * NI];
  __shared__ int32_t hist[8 * LPR * NI];
  __shared__ double sl[kDirectThreads / 64];
  const int s = blockIdx.x;
  uint32_t r0, r1;
  segment_bounds(offs, s, rows, r0, r1);
  sum_rows<T, LPR, NI, SIGMOID, kDirectThreads>(z, ld, E, ids, ids_ld, K, r0, r1, part, hist);
  double term = 0.0;
  const int c = threadIdx.x;  // E <= 1024: one column per thread
  if (c < E) {
    const float p = part[0][c];
    psum[static_cast<int64_t>(s) * E + c] = p;
    counts[static_cast<int64_t>(s) * E + c] = hist[c];
    term = static_cast<double>(p) * hist[c];
  }
  write_loss<kDirectThreads>(term, balance_scale(coeff, E, K, r1 - r0), loss + s, sl);
}

// One workgroup per segment: `strips` threads per expert (1024 over E rounded up
// to a power of two) add the segment's slots, then the loss.
__global__ __launch_bounds__(kFoldThreads) void router_fold_kernel(const float* __restrict__ slot_p,
                                                                   const int32_t* __restrict__ slot_c,
                                                                   const int32_t* __restrict__ table,
                                                                   const int32_t* __restrict__ offs, uint32_t rows,
                                                                   int E, int K, int log_cols, double coeff,
                                                                   float* __restrict__ psum,
                                                                   int32_t* __restrict__ counts,
                                                                   float* __restrict__ loss) {
  constexpr int kRound = 16;  // slots of a strip in flight together
  __shared__ double sp[kFoldThreads];
  __shared__ int32_t sc[kFoldThreads];
  __shared__ double sl[kFoldThreads / 64];
  const int s = blockIdx.x, cols = 1 << log_cols, strips = kFoldThreads >> log_cols;
  const int c = threadIdx.x & (cols - 1), strip = threadIdx.x >> log_cols;
  const int t0 = table[s], t1 = table[s + 1];
  uint32_t b0, b1;
  segment_bounds(offs, s, rows, b0, b1);
  const double scale = balance_scale(coeff, E, K, b1 - b0);
  double p = 0.0;
  int32_t n = 0;
  const int cc = c < E ? c : 0;
  for (int t = t0 + strip; t < t1; t += kRound * strips) {
    float v[kRound];
    int32_t k[kRound];
#pragma unroll
    for (int i = 0; i < kRound; ++i) {  // past the last tile: the strip's first one again, and not added
      const int64_t at = static_cast<int64_t>(t + i * strips < t1 ? t + i * strips : t) * E + cc;
      v[i] = slot_p[at];
      k[i] = slot_c[at];
    }
#pragma unroll
    for (int i = 0; i < kRound; ++i) {
      const bool in = t + i * strips < t1;
      p += in ? v[i] : 0.0f;
      n += in ? k[i] : 0;
    }
  }
  sp[threadIdx.x] = p;
  sc[threadIdx.x] = n;
  __syncthreads();
  double term = 0.0;
  if (strip == 0 && c < E) {
    for (int i = 1; i < strips; ++i) {
      p += sp[(i << log_cols) + c];
      n += sc[(i << log_cols) + c];
    }
    psum[static_cast<int64_t>(s) * E + c] = static_cast<float>(p);
    counts[static_cast<int64_t>(s) * E + c] = n;
    term = p * n;
  }
  write_loss<kFoldThreads>(term, scale, loss + s, sl);
}

template <typename T, int LPR, int NI, bool SIGMOID>
__global__ __launch_bounds__(kBwdThreads) void router_bwd_kernel(T* __restrict__ dz, int64_t ld_d,
                                                                 const T* __restrict__ z, int64_t ld, uint32_t rows,
                                                                 int E, int K, const int32_t* __restrict__ offs,
                                                                 int S, int log_bt, const int32_t* __restrict__ counts,
                                                                 const float* __restrict__ dloss, double coeff) {
  constexpr int RPW = 64 / LPR, W = kBwdThreads / 64, kBwdAhead = bwd_ahead(NI);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int seg;
  uint32_t r0, r1, s0, s1;
  if (!segment_tile<kScanBatch>(offs, S, rows, log_bt, blockIdx.x, seg, r0, r1, s0, s1)) return;
  const float g = static_cast<float>(balance_scale(coeff, E, K, s1 - s0) * dloss[seg]);
  const int sub = lane / LPR, l = lane % LPR;
  // c_e less the mean count: the gradient does not change (sum p = 1), and the
  // difference c_e - sum p c keeps its digits when the experts are nearly balanced
  const int32_t ref = static_cast<int32_t>(static_cast<uint32_t>(K) * (s1 - s0) / static_cast<uint32_t>(E));
  Cols<LPR == 1> c[NI];
  float n[NI][8];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    c[i].set((i * LPR + l) * 8, E, 8 * LPR * NI);
    Raw8<float> raw;  // whole numbers, moved as bits
    load_cols(raw, reinterpret_cast<const float*>(counts) + static_cast<int64_t>(seg) * E, c[i]);
    raw.get(n[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) n[i][j] = c[i].own(j) ? static_cast<float>(__float_as_int(n[i][j]) - ref) : 0.0f;
  }
  for (uint32_t r = r0 + wave * RPW; r < r1; r += kBwdAhead * W * RPW) {
    float v[kBwdAhead][NI][8];
    load_rows<T, LPR, NI, kBwdAhead>(z, ld, r + sub, W * RPW, r0, r1, c, v);
#pragma unroll
    for (int a = 0; a < kBwdAhead; ++a) {
      const uint32_t row = r + sub + a * W * RPW;
      float e[NI][8], q[NI][8];
      const float inv = row_scores<LPR, NI, SIGMOID, true>(v[a], e, q);
      float mean = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) mean = __builtin_fmaf(e[i][j], n[i][j], mean);
      const float gi = g * inv, gm = lanes_sum<LPR>(mean) * inv * gi;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          d[j] = e[i][j] * __builtin_fmaf(n[i][j], gi, -gm);
          if (SIGMOID) d[j] *= q[i][j];
        }
        if (row < r1) store_cols(dz + static_cast<int64_t>(row) * ld_d, c[i], d);
      }
    }
  }
}

int64_t max_tiles(int64_t T, int64_t S, int log_bt) { return ceil_div(T, int64_t(1) << log_bt) + S; }

int columns_per_lane(int64_t E) { return E > 16 ? 16 : 8; }
int64_t lanes_per_row(int64_t E) {
  int64_t lpr = 1;
  while (lpr * columns_per_lane(E) < E) lpr *= 2;
  return lpr;
}

// Rows per tile, a power of two from the shape alone: about `target` tiles, but
// no fewer rows than the workgroup's waves take in one step of `ahead` rows per
// lane group. A step at 65536 x 256 takes 33.2 us with 512 and 1024 tiles (forward,
// backward), 34.5 with 256 and 1024, 36.2 with 1024 and 2048, 35.9 with 512 and 512.
int tile_log(int64_t T, int64_t E, int threads, int (*ahead)(int), int64_t target) {
  const int64_t step = threads / lanes_per_row(E) * ahead(columns_per_lane(E) / 8);
  int lg = 0;
  while ((int64_t(1) << lg) < step || (T >> lg) > target) ++lg;
  return lg;
}
int fwd_log(int64_t T, int64_t E) { return tile_log(T, E, kFwdThreads, fwd_ahead, 512); }
int bwd_log(int64_t T, int64_t E) { return tile_log(T, E, kBwdThreads, bwd_ahead, 1024); }

// A call is summed by one workgroup per segment, in one launch, where that takes
// no longer than the second launch and its slots. What such a workgroup does is
// steps (its lanes' rows at a time, one memory latency each) and slots (LDS atomics
// on few addresses); the host knows S but not the segments, so a mean segment is
// held to 4 steps and 8192 slots and the longest possible one to 16 steps, 2^17
// logits and 32768 slots (16384 x 2, K 2 in one of several segments, the worst of
// these: 29 us against 19).
// GPU time of one and of two launches (in a graph; outside, two take 11 us of the
// host), us, float32:
//   48 x 8, K 2, S 3        5.3  10.2     2048 x 32, K 4, S 1    11.0   9.6
//   4096 x 8, K 2, S 1      8.0  10.4     4096 x 32, K 4, S 1    15.9   9.9
//   8192 x 8, K 2, S 1     11.0  10.3     4096 x 32, K 4, S 8     8.2   9.9
//   16384 x 8, K 2, S 1    17.7  10.4     256 x 256, K 8, S 1     8.4   8.4
//   16384 x 8, K 2, S 8     6.7  10.8     512 x 256, K 8, S 1    12.3   8.4
//   16384 x 8, K 8, S 1    37.9  12.1     65536 x 2, K 2, S 1   100.9  19.4
bool direct(int64_t T, int64_t E, int64_t K, int64_t S) {
  const int64_t rows = kDirectThreads / lanes_per_row(E), mean = ceil_div(T, S < 1 ? 1 : S);
  return ceil_div(mean, rows) <= 4 && mean * K <= 8192 && ceil_div(T, rows) <= 16 && T * E <= 131072 &&
         T * K <= 32768;
}

struct RouterWs {
  size_t table, p, c, total;
};
RouterWs layout(int64_t T, int64_t E, int64_t S) {
  RouterWs w;
  const size_t n = static_cast<size_t>(max_tiles(T, S, fwd_log(T, E)) * E) * 4;
  w.table = DET_WS_HEADER_BYTES;
  w.p = w.table + align_up(static_cast<size_t>(S + 1) * 4, 256);
  w.c = w.p + align_up(n, 256);
  w.total = w.c + align_up(n, 256);
  return w;
}

int check_sizes(const char* what, int64_t T, int64_t E, int64_t K, int64_t S) {
  if (T < 0 || S < 0) return set_error(DET_ERR_INVALID_ARG, "%s: T and S must be >= 0", what);
  if (E < 1 || K < 1) return set_error(DET_ERR_INVALID_ARG, "%s: E and K must be >= 1", what);
  if (E > 1024) return set_error(DET_ERR_UNSUPPORTED, "%s: E must be <= 1024, got %lld", what, (long long)E);
  if (K > 65536 || T > (int64_t(1) << 30) || T * K >= (int64_t(1) << 31))
    return set_error(DET_ERR_UNSUPPORTED, "%s: T * K must be < 2^31 (T <= 2^30, K <= 65536)", what);
  if (S > 65535) return set_error(DET_ERR_UNSUPPORTED, "%s: S must be <= 65535", what);
  return DET_OK;
}

int check_call(const char* what, int dtype, int score, double coeff, int64_t T, int64_t E, int64_t ld) {
  if (int s = check_float_dtype(what, dtype)) return s;
  if (score != DET_SCORE_SOFTMAX && score != DET_SCORE_SIGMOID)
    return set_error(DET_ERR_INVALID_ARG, "%s: score must be DET_SCORE_SOFTMAX or DET_SCORE_SIGMOID, got %d", what,
                     score);
  if (!(coeff - coeff == 0.0)) return set_error(DET_ERR_INVALID_ARG, "%s: coeff must be finite", what);
  if (T && ld < E) return set_error(DET_ERR_INVALID_ARG, "%s: a row stride of the logits is < E", what);
  if (T && ld > (int64_t(1) << 44) / T) return set_error(DET_ERR_UNSUPPORTED, "%s: tensor too large", what);
  return DET_OK;
}

}  // namespace
}  // namespace detgrad

using namespace detgrad;

// LPR x NI by E (eight columns per lane and NI), the element type and the score.
#define DET_ROUTER_BY_E(F, TYPE, SIG)          \
  if (E <= 8) { F(TYPE, SIG, 1, 1) }           \
  else if (E <= 16) { F(TYPE, SIG, 2, 1) }     \
  else if (E <= 32) { F(TYPE, SIG, 2, 2) }     \
  else if (E <= 64) { F(TYPE, SIG, 4, 2) }     \
  else if (E <= 128) { F(TYPE, SIG, 8, 2) }    \
  else if (E <= 256) { F(TYPE, SIG, 16, 2) }   \
  else if (E <= 512) { F(TYPE, SIG, 32, 2) }   \
  else { F(TYPE, SIG, 64, 2) }
#define DET_ROUTER_DISPATCH(F)                                                 \
  if (dtype == DET_BF16) {                                                     \
    if (score == DET_SCORE_SIGMOID) { DET_ROUTER_BY_E(F, uint16_t, true) }     \
    else { DET_ROUTER_BY_E(F, uint16_t, false) }                               \
  } else {                                                                     \
    if (score == DET_SCORE_SIGMOID) { DET_ROUTER_BY_E(F, float, true) }        \
    else { DET_ROUTER_BY_E(F, float, false) }                                  \
  }

extern "C" int det_router_balance_workspace_size(int64_t T, int64_t E, int64_t K, int64_t S, size_t* bytes) {
  if (!bytes) return set_error(DET_ERR_INVALID_ARG, "router_balance: bytes is NULL");
  if (int s = check_sizes("router_balance", T, E, K, S)) return s;
  *bytes = S == 0 || direct(T, E, K, S) ? 0 : layout(T, E, S).total;
  return ok();
}

extern "C" int det_router_balance(const void* logits, int64_t ld, int dtype, const int32_t* ids, int64_t ids_ld,
                                  int64_t T, int64_t E, int64_t K, const int32_t* offs, int64_t S, int score,
                                  double coeff, int32_t* counts, float* prob_sum, float* loss, void* ws,
                                  size_t ws_bytes, void* stream) {
  const char* what = "router_balance";
  if (int s = check_sizes(what, T, E, K, S)) return s;
  if (int s = check_call(what, dtype, score, coeff, T, E, ld)) return s;
  if (S == 0) return ok();  // no segments: no outputs
  if (!offs || !counts || !prob_sum || !loss || (T && (!logits || !ids)))
    return set_error(DET_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if (T && ids_ld < K) return set_error(DET_ERR_INVALID_ARG, "%s: ids row stride < K", what);
  if (T && ids_ld > (int64_t(1) << 44) / T) return set_error(DET_ERR_UNSUPPORTED, "%s: tensor too large", what);
  const bool one = direct(T, E, K, S);
  const RouterWs w = layout(T, E, S);
  if (int s = check_workspace(ws, ws_bytes, one ? 0 : w.total)) return s;
  const size_t es = dtype_size(dtype);
  const Buf outs[] = {{"counts", range1d(counts, S * E * 4)},
                      {"prob_sum", range1d(prob_sum, S * E * 4)},
                      {"loss", range1d(loss, S * 4)},
                      {"the workspace", range1d(one ? nullptr : ws, ws_bytes)}};
  const Buf ins[] = {buf_rows("logits", logits, T, E, ld, es),
                     buf_rows("ids", ids, T, K, ids_ld, 4),
                     {"offs", range1d(offs, (S + 1) * 4)}};
  if (int s = check_buffers(what, outs, 4, ins, 3)) return s;
  const hipStream_t st = as_stream(stream);
  char* b = static_cast<char*>(ws);
  auto* table = one ? nullptr : reinterpret_cast<int32_t*>(b + w.table);
  auto* sp = one ? nullptr : reinterpret_cast<float*>(b + w.p);
  auto* sc = one ? nullptr : reinterpret_cast<int32_t*>(b + w.c);
  const int lg = fwd_log(T, E);
  const dim3 grid(static_cast<uint32_t>(one ? S : max_tiles(T, S, lg)));
#define DET_ROUTER_FWD(TYPE, SIG, LPR, NI)                                                                       \
  {                                                                                                              \
    if (one)                                                                                                     \
      hipLaunchKernelGGL((router_direct_kernel<TYPE, LPR, NI, SIG>), grid, dim3(kDirectThreads), 0, st,          \
                         static_cast<const TYPE*>(logits), ld, (uint32_t)T, (int)E, ids, ids_ld, (int)K, offs,   \
                         coeff, prob_sum, counts, loss);                                                         \
    else                                                                                                         \
      hipLaunchKernelGGL((router_tile_kernel<TYPE, LPR, NI, SIG>), grid, dim3(kFwdThreads), 0, st,               \
                         static_cast<const TYPE*>(logits), ld, (uint32_t)T, (int)E, ids, ids_ld, (int)K, offs,   \
                         (int)S, lg, sp, sc, table);                                                             \
  }
  DET_ROUTER_DISPATCH(DET_ROUTER_FWD)
#undef DET_ROUTER_FWD
  if (!one) {
    int log_cols = 0;
    while ((1 << log_cols) < E) ++log_cols;
    hipLaunchKernelGGL(router_fold_kernel, dim3(static_cast<uint32_t>(S)), dim3(kFoldThreads), 0, st, sp, sc, table,
                       offs, (uint32_t)T, (int)E, (int)K, log_cols, coeff, prob_sum, counts, loss);
  }
  return check_launch("det_router_balance");
}

extern "C" int det_router_balance_bwd(void* dlogits, int64_t ld_d, const void* logits, int64_t ld, int dtype, int64_t T,
                                      int64_t E, int64_t K, const int32_t* offs, int64_t S, const int32_t* counts,
                                      const float* dloss, int score, double coeff, void* stream) {
  const char* what = "router_balance_bwd";
  if (int s = check_sizes(what, T, E, K, S)) return s;
  if (int s = check_call(what, dtype, score, coeff, T, E, ld)) return s;
  if (int s = check_call(what, dtype, score, coeff, T, E, ld_d)) return s;
  if (T == 0 || S == 0) return ok();  // no rows in any segment: dlogits unchanged
  if (!dlogits || !logits || !offs || !counts || !dloss)
    return set_error(DET_ERR_INVALID_ARG, "%s: NULL pointer", what);
  const size_t es = dtype_size(dtype);
  const Buf outs[] = {buf_rows("dlogits", dlogits, T, E, ld_d, es)};
  const Buf ins[] = {buf_rows("logits", logits, T, E, ld, es),
                     {"offs", range1d(offs, (S + 1) * 4)},
                     {"counts", range1d(counts, S * E * 4)},
                     {"dloss", range1d(dloss, S * 4)}};
  if (int s = check_buffers(what, outs, 1, ins, 4)) return s;
  const hipStream_t st = as_stream(stream);
  const int lg = bwd_log(T, E);
  const dim3 grid(static_cast<uint32_t>(max_tiles(T, S, lg)));
#define DET_ROUTER_BWD(TYPE, SIG, LPR, NI)                                                                       \
  hipLaunchKernelGGL((router_bwd_kernel<TYPE, LPR, NI, SIG>), grid, dim3(kBwdThreads), 0, st,                    \
                     static_cast<TYPE*>(dlogits), ld_d, static_cast<const TYPE*>(logits), ld, (uint32_t)T,       \
                     (int)E, (int)K, offs, (int)S, lg, counts, dloss, coeff);
  DET_ROUTER_DISPATCH(DET_ROUTER_BWD)
#undef DET_ROUTER_BWD
  return check_launch("det_router_balance_bwd");
}
