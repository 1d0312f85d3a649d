// det_router_balance / det_router_balance_bwd: the router's load-balancing loss
// with its per-expert counts and score sums, and the gradient of its logits.
//
//   p[t]         = softmax(z[t]), or sigmoid(z[t]) / sum sigmoid(z[t]) (the softmax of log sigmoid(z))
//   counts[s][e] = slots (t, k) of segment s with ids[t][k] == e
//   P[s][e]      = sum of p[t][e] over the tokens of segment s
//   loss[s]      = coeff E / (K N_s^2) sum_e counts[s][e] P[s][e]
//   dz[t][e]     = dloss[s] coeff E / (K N_s^2) p_e (c_e - sum_j p_j c_j)   [(1 - sigmoid(z_e)) for the sigmoid score]
//
// Layout: a row of E logits sits in LPR lanes of eight consecutive columns (one
// or two 16-byte loads per lane), 64 / LPR rows per wave and step, so the
// softmax's maximum and sum are a few lane exchanges and every lane keeps the
// running P of its own columns in registers.
//
// Order of P (no atomics): a tile of rows of one segment belongs to one
// workgroup; lane group g of wave w adds its rows of the tile in ascending
// order, the lane groups of a wave meet in an adjacent tree, the waves left to
// right, and the tile's sum is one float32 slot. The fold adds a segment's
// slots in float64, in tile order per strip and the strips in order. Counts are
// whole numbers, so their LDS atomics have one result.
//
// Both kernels are bound by reading the logits (and writing dz), and at small
// sizes by the launches.
#include "rowops.hpp"
#include "segtiles.hpp"

namespace detgrad {
namespace {

constexpr int kFwdThreads = 512, kBwdThreads = 256, kFoldThreads = 1024;

__device__ __forceinline__ float log_sigmoid(float z) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(z) * kLog2e);
  return fminf(z, 0.0f) - kLn2 * __builtin_amdgcn_logf(1.0f + e);
}

// The row's unnormalised scores e (0 past the row's end and in a row whose
// logits are all -inf) and 1 / their sum (0 for such a row). z: the logits,
// -inf past the end.
template <int LPR, int NI>
__device__ __forceinline__ float row_scores(const float (&z)[NI][8], bool sigmoid, float (&e)[NI][8], float& sum) {
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      e[i][j] = sigmoid ? log_sigmoid(z[i][j]) : z[i][j];
      m = fmaxf(m, e[i][j]);
    }
  m = lanes_max<LPR>(m);
  m = m == -__builtin_inff() ? 0.0f : m;  // nothing but -inf: every score is exp(-inf) = 0 (and a NaN stays one)
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      e[i][j] = exp_e(e[i][j] - m);
      s += e[i][j];
    }
  sum = lanes_sum<LPR>(s);
  return sum == 0.0f ? 0.0f : 1.0f / sum;
}

template <typename T, int LPR, int NI>
__global__ __launch_bounds__(kFwdThreads) void router_tile_kernel(const T* __restrict__ z, int64_t ld, uint32_t rows,
                                                                  int E, const int32_t* __restrict__ ids,
                                                                  int64_t ids_ld, int K,
                                                                  const int32_t* __restrict__ offs, int S, int log_bt,
                                                                  int sigmoid, float* __restrict__ slot_p,
                                                                  int32_t* __restrict__ slot_c,
                                                                  int32_t* __restrict__ table) {
  constexpr int RPW = 64 / LPR, W = kFwdThreads / 64, COLS = 8 * LPR * NI;
  __shared__ float part[W][COLS];
  __shared__ int32_t hist[COLS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (blockIdx.x == 0 && wave == 0) write_tile_table(offs, S, rows, log_bt, table);
  int seg;
  uint32_t r0, r1;
  if (!tile_of(offs, S, rows, log_bt, blockIdx.x, seg, r0, r1)) return;  // the grid covers the worst case
  for (int i = threadIdx.x; i < COLS; i += kFwdThreads) hist[i] = 0;
  __syncthreads();
  const uint32_t slots = (r1 - r0) * static_cast<uint32_t>(K);  // < 2^31 (checked by the host)
  for (uint32_t i = threadIdx.x; i < slots; i += kFwdThreads) {
    const uint32_t r = i / static_cast<uint32_t>(K);
    const int32_t id = ids[static_cast<int64_t>(r0 + r) * ids_ld + (i - r * K)];
    if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
  }
  float acc[NI][8] = {};
  const int sub = lane / LPR, l = lane % LPR;
  for (uint32_t r = r0 + wave * RPW; r < r1; r += W * RPW) {
    const bool in = r + sub < r1;
    float v[NI][8], e[NI][8], sum;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int col = (i * LPR + l) * 8;
      load8(z + static_cast<int64_t>(in ? r + sub : r) * ld + col, in ? E - col : 0, -__builtin_inff(), v[i]);
    }
    const float inv = row_scores<LPR, NI>(v, sigmoid, e, sum);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] += e[i][j] * inv;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int d = LPR; d < 64; d <<= 1) acc[i][j] += __shfl_xor(acc[i][j], d);
      if (sub == 0) part[wave][(i * LPR + l) * 8 + j] = acc[i][j];
    }
  __syncthreads();
  for (int c = threadIdx.x; c < E; c += kFwdThreads) {
    float s = part[0][c];
#pragma unroll
    for (int w = 1; w < W; ++w) s += part[w][c];
    slot_p[static_cast<int64_t>(blockIdx.x) * E + c] = s;
    slot_c[static_cast<int64_t>(blockIdx.x) * E + c] = hist[c];
  }
}

// b_s for every lane: the running maximum of the clamped offsets up to s.
__device__ __forceinline__ uint32_t segment_bound(const int32_t* __restrict__ offs, int s, uint32_t rows) {
  uint32_t b = 0;
  for (int i = threadIdx.x & 63; i <= s; i += 64) b = umax(b, clamp_off(offs[i], rows));
  return lane_value(scan_max(b), 63);
}

__device__ __forceinline__ double balance_scale(double coeff, int E, int K, uint32_t n) {
  return n == 0 ? 0.0 : coeff * E / (static_cast<double>(K) * n * n);
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
  __shared__ double sp[kFoldThreads];
  __shared__ int32_t sc[kFoldThreads];
  __shared__ double sl[kFoldThreads / 64];
  const int s = blockIdx.x, cols = 1 << log_cols, strips = kFoldThreads >> log_cols;
  const int c = threadIdx.x & (cols - 1), strip = threadIdx.x >> log_cols;
  const int t0 = table[s], t1 = table[s + 1];
  double p = 0.0;
  int32_t n = 0;
  if (c < E)
    for (int t = t0 + strip; t < t1; t += 8 * strips) {
      float v[8];
      int32_t k[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int tt = t + i * strips;
        v[i] = tt < t1 ? slot_p[static_cast<int64_t>(tt) * E + c] : 0.0f;
        k[i] = tt < t1 ? slot_c[static_cast<int64_t>(tt) * E + c] : 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p += v[i];
        n += k[i];
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
  for (int d = 1; d < 64; d <<= 1) term += __shfl_xor(term, d);
  if ((threadIdx.x & 63) == 0) sl[threadIdx.x >> 6] = term;
  __syncthreads();
  if (threadIdx.x < 64) {
    const uint32_t n_s = segment_bound(offs, s + 1, rows) - segment_bound(offs, s, rows);
    double tot = 0.0;
    for (int w = 0; w < kFoldThreads / 64; ++w) tot += sl[w];
    if (threadIdx.x == 0) loss[s] = static_cast<float>(balance_scale(coeff, E, K, n_s) * tot);
  }
}

template <typename T, int LPR, int NI>
__global__ __launch_bounds__(kBwdThreads) void router_bwd_kernel(T* __restrict__ dz, int64_t ld_d,
                                                                 const T* __restrict__ z, int64_t ld, uint32_t rows,
                                                                 int E, int K, const int32_t* __restrict__ offs,
                                                                 int S, int log_bt, const int32_t* __restrict__ counts,
                                                                 const float* __restrict__ dloss, double coeff,
                                                                 int sigmoid) {
  constexpr int RPW = 64 / LPR, W = kBwdThreads / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int seg;
  uint32_t r0, r1, s0, s1;
  if (!segment_tile(offs, S, rows, log_bt, blockIdx.x, seg, r0, r1, s0, s1)) return;
  const float g = static_cast<float>(balance_scale(coeff, E, K, s1 - s0) * dloss[seg]);
  const int sub = lane / LPR, l = lane % LPR;
  // c_e less the mean count: the gradient does not change (sum p = 1), and the
  // difference c_e - sum p c keeps its digits when the experts are nearly balanced
  const int64_t ref = static_cast<int64_t>(K) * (s1 - s0) / E;
  float c[NI][8];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = (i * LPR + l) * 8 + j;
      c[i][j] = e < E ? static_cast<float>(counts[static_cast<int64_t>(seg) * E + e] - ref) : 0.0f;
    }
  for (uint32_t r = r0 + wave * RPW; r < r1; r += W * RPW) {
    const bool in = r + sub < r1;
    const int64_t row = in ? r + sub : r;
    float v[NI][8], e[NI][8], sum;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int col = (i * LPR + l) * 8;
      load8(z + row * ld + col, in ? E - col : 0, -__builtin_inff(), v[i]);
    }
    const float inv = row_scores<LPR, NI>(v, sigmoid, e, sum);
    float mean = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) mean += e[i][j] * c[i][j];
    mean = lanes_sum<LPR>(mean) * inv;
    const float gi = g * inv;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int col = (i * LPR + l) * 8;
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        d[j] = gi * e[i][j] * (c[i][j] - mean);
        if (sigmoid) d[j] = d[j] / (1.0f + exp_e(v[i][j]));
      }
      if (in) store8(dz + row * ld_d + col, E - col, d);
    }
  }
}

int64_t max_tiles(int64_t T, int64_t S, int log_bt) { return ceil_div(T, int64_t(1) << log_bt) + S; }

// Rows per tile, a power of two from the shape alone: about `target` tiles, but
// no fewer rows than one step of the workgroup's waves takes.
int tile_log(int64_t T, int64_t E, int threads, int64_t target) {
  int64_t lpr = 1;
  while (lpr * 8 < E && lpr < 64) lpr *= 2;
  const int64_t step = threads / 64 * (64 / lpr);
  int lg = 0;
  while ((int64_t(1) << lg) < step || (T >> lg) > target) ++lg;
  return lg;
}
int fwd_log(int64_t T, int64_t E) { return tile_log(T, E, kFwdThreads, 256); }
int bwd_log(int64_t T, int64_t E) { return tile_log(T, E, kBwdThreads, 2048); }

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

// LPR x NI by E (eight columns per lane): calls F<LPR, NI>.
#define DET_ROUTER_BY_E(F)    \
  if (E <= 8) F(1, 1)         \
  else if (E <= 16) F(2, 1)   \
  else if (E <= 32) F(4, 1)   \
  else if (E <= 64) F(8, 1)   \
  else if (E <= 128) F(16, 1) \
  else if (E <= 256) F(32, 1) \
  else if (E <= 512) F(64, 1) \
  else F(64, 2)

extern "C" int det_router_balance_workspace_size(int64_t T, int64_t E, int64_t K, int64_t S, size_t* bytes) {
  if (!bytes) return set_error(DET_ERR_INVALID_ARG, "router_balance: bytes is NULL");
  if (int s = check_sizes("router_balance", T, E, K, S)) return s;
  *bytes = S == 0 ? 0 : layout(T, E, S).total;
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
  const RouterWs w = layout(T, E, S);
  if (int s = check_workspace(ws, ws_bytes, w.total)) return s;
  const size_t es = dtype_size(dtype);
  const Buf outs[] = {{"counts", range1d(counts, S * E * 4)},
                      {"prob_sum", range1d(prob_sum, S * E * 4)},
                      {"loss", range1d(loss, S * 4)},
                      {"the workspace", range1d(ws, ws_bytes)}};
  const Buf ins[] = {{"logits", range2d(logits, T, E, ld, es)},
                     {"ids", range2d(ids, T, K, ids_ld, 4)},
                     {"offs", range1d(offs, (S + 1) * 4)}};
  if (int s = check_overlaps(what, outs, 4, ins, 3)) return s;
  const hipStream_t st = as_stream(stream);
  char* b = static_cast<char*>(ws);
  auto* table = reinterpret_cast<int32_t*>(b + w.table);
  auto* sp = reinterpret_cast<float*>(b + w.p);
  auto* sc = reinterpret_cast<int32_t*>(b + w.c);
  const int lg = fwd_log(T, E);
  const dim3 grid(static_cast<uint32_t>(max_tiles(T, S, lg)));
  const int sg = score == DET_SCORE_SIGMOID;
#define DET_ROUTER_FWD(LPR, NI)                                                                                       \
  {                                                                                                                   \
    if (dtype == DET_BF16)                                                                                            \
      hipLaunchKernelGGL((router_tile_kernel<uint16_t, LPR, NI>), grid, dim3(kFwdThreads), 0, st,                     \
                         static_cast<const uint16_t*>(logits), ld, (uint32_t)T, (int)E, ids, ids_ld, (int)K, offs,    \
                         (int)S, lg, sg, sp, sc, table);                                                              \
    else                                                                                                              \
      hipLaunchKernelGGL((router_tile_kernel<float, LPR, NI>), grid, dim3(kFwdThreads), 0, st,                        \
                         static_cast<const float*>(logits), ld, (uint32_t)T, (int)E, ids, ids_ld, (int)K, offs,       \
                         (int)S, lg, sg, sp, sc, table);                                                              \
  }
  DET_ROUTER_BY_E(DET_ROUTER_FWD)
#undef DET_ROUTER_FWD
  int log_cols = 0;
  while ((1 << log_cols) < E) ++log_cols;
  hipLaunchKernelGGL(router_fold_kernel, dim3(static_cast<uint32_t>(S)), dim3(kFoldThreads), 0, st, sp, sc, table, offs,
                     (uint32_t)T, (int)E, (int)K, log_cols, coeff, prob_sum, counts, loss);
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
  const Buf outs[] = {{"dlogits", range2d(dlogits, T, E, ld_d, es)}};
  const Buf ins[] = {{"logits", range2d(logits, T, E, ld, es)},
                     {"offs", range1d(offs, (S + 1) * 4)},
                     {"counts", range1d(counts, S * E * 4)},
                     {"dloss", range1d(dloss, S * 4)}};
  if (int s = check_overlaps(what, outs, 1, ins, 4)) return s;
  const hipStream_t st = as_stream(stream);
  const int lg = bwd_log(T, E);
  const dim3 grid(static_cast<uint32_t>(max_tiles(T, S, lg)));
  const int sg = score == DET_SCORE_SIGMOID;
#define DET_ROUTER_BWD(LPR, NI)                                                                                       \
  {                                                                                                                   \
    if (dtype == DET_BF16)                                                                                            \
      hipLaunchKernelGGL((router_bwd_kernel<uint16_t, LPR, NI>), grid, dim3(kBwdThreads), 0, st,                      \
                         static_cast<uint16_t*>(dlogits), ld_d, static_cast<const uint16_t*>(logits), ld,             \
                         (uint32_t)T, (int)E, (int)K, offs, (int)S, lg, counts, dloss, coeff, sg);                    \
    else                                                                                                              \
      hipLaunchKernelGGL((router_bwd_kernel<float, LPR, NI>), grid, dim3(kBwdThreads), 0, st,                         \
                         static_cast<float*>(dlogits), ld_d, static_cast<const float*>(logits), ld, (uint32_t)T,      \
                         (int)E, (int)K, offs, (int)S, lg, counts, dloss, coeff, sg);                                 \
  }
  DET_ROUTER_BY_E(DET_ROUTER_BWD)
#undef DET_ROUTER_BWD
  return check_launch("det_router_balance_bwd");
}
