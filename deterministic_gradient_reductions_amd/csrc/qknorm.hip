// det_qk_norm / det_qk_norm_bwd: the norm of every head of the queries and keys, its
// weights, and the rotation of channel pairs by position, in one pass.
//
//   n = w x rstd,  rstd = 1 / sqrt(mean(x^2) + eps)   (L2: the sum; none: 1)
//   (y_a, y_b) = (n_a cos - n_b sin, n_b cos + n_a sin),  angle = pos[axis[p]] * inv_freq[p] of pair p
//
// and back, with d = dy turned by the opposite angle:
//
//   dw += sum d x rstd,  u = w d:  dx = rstd (u - xh mean(u xh)),  xh = x rstd   (L2: the sum; none: dx = u)
//
// A head's row lies in the fewest lanes that hold it at eight channel pairs each (a
// power of two), so a pair is in one lane and a row's sums are lane exchanges. A
// lane's pairs are two runs of eight channels (pairs of halves) or one of sixteen
// (neighbours, and the channels behind the rotated ones), so rows are read and written
// sixteen bytes at a time. The angles of a token serve all its heads: a workgroup
// forms the sines of its tokens once, in LDS, from the product of position and
// frequency in float64 (a float32 product of a position of 10^6 is off by 0.03 of a
// radian). The backward needs no value of the forward but x: it forms rstd again.
//
// The parameter gradients are ordered column sums: every lane adds its rows in order,
// a workgroup its lanes' sums, and a fold the workgroups' in float64; no atomics.
//
// Both are bound by the [T, heads, D] tensors.
#include "delta.hpp"

namespace detgrad {
namespace {

constexpr int kThreads = 256, kMaxD = 1024, kTurns = 2048, kFoldWaves = 16;
enum Mode { kHalves = 0, kNeighbours = 1, kMixed = 2, kEither = 3 };

// What a launch works by. pairs [0, half) are turned.
struct QkPlan {
  int64_t T;
  int D, half, lanes, tokens, groups, norm;  // lanes of a row, tokens of a workgroup's turn, rows side by side
  bool halves, past;
  float eps, inv;
  const int32_t *pos, *axis;
  int64_t pos_ld;
  int axes;
  const float* inv_freq;
};

// Channel of side `s` of pair p, or D where there is none.
__device__ __forceinline__ int channel(const QkPlan& P, int p, int s) {
  const int d = P.halves && p < P.half ? p + s * P.half : 2 * p + s;
  return 2 * p < P.D + 1 && d < P.D ? d : P.D;
}

// A lane's eight pairs of a row.
struct Spot {
  int p0, off[2];  // first pair; first channels of the two runs of eight
  bool live;       // there are any of them
  bool fast;       // both runs lie in the row as they stand
  bool split;      // the runs are the two sides (else sixteen neighbours)
};
__device__ __forceinline__ Spot spot_of(const QkPlan& P) {
  Spot s;
  s.p0 = 8 * (threadIdx.x & (P.lanes - 1));
  s.split = P.halves && s.p0 < P.half;
  s.off[0] = s.split ? s.p0 : 2 * s.p0;
  s.off[1] = s.split ? s.p0 + P.half : 2 * s.p0 + 8;
  s.live = 2 * s.p0 < P.D;
  s.fast = s.split ? s.p0 + 8 <= P.half : 2 * s.p0 + 16 <= P.D;
  if (!s.live) s.off[0] = s.off[1] = 0;  // (loaded, not used)
  return s;
}

// The lane's pairs of a row as they are in memory: in the fast case one of the two forms
// below, else element by element; loads under a branch of the lane's own would be waited
// for one by one. What a lane has not is zero.
template <typename T, int MODE>
struct Row {
  Raw8<T> r[2];
  T slow[MODE == kMixed ? 16 : 1];
  __device__ __forceinline__ void load(const T* row, const QkPlan& P, const Spot& s) {
    if (MODE != kMixed || s.fast) {
      r[0].load(row + s.off[0]);
      r[1].load(row + s.off[1]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = channel(P, s.p0 + j, e);
          slow[MODE == kMixed ? 2 * j + e : 0] = row[d < P.D ? d : 0];
        }
    }
  }
  __device__ __forceinline__ void get(const QkPlan& P, const Spot& s, float (&a)[8], float (&b)[8]) const {
    float x[8], y[8];
    r[0].get(x);
    r[1].get(y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float na = j < 4 ? x[2 * (j & 3)] : y[2 * (j & 3)], nb = j < 4 ? x[2 * (j & 3) + 1] : y[2 * (j & 3) + 1];
      if (MODE == kHalves) {
        a[j] = x[j];
        b[j] = y[j];
      } else if (MODE == kNeighbours) {
        a[j] = na;
        b[j] = nb;
      } else if (MODE == kEither) {
        a[j] = s.split ? x[j] : na;
        b[j] = s.split ? y[j] : nb;
      } else {
        a[j] = s.fast ? (s.split ? x[j] : na) : channel(P, s.p0 + j, 0) < P.D ? to_f32(slow[2 * j]) : 0.0f;
        b[j] = s.fast ? (s.split ? y[j] : nb) : channel(P, s.p0 + j, 1) < P.D ? to_f32(slow[2 * j + 1]) : 0.0f;
      }
      if (MODE != kMixed && !s.live) a[j] = b[j] = 0.0f;
    }
  }
};

template <int MODE, typename T>
__device__ __forceinline__ void put_row(T* row, const QkPlan& P, const Spot& s, const float (&a)[8], const float (&b)[8]) {
  if (MODE != kMixed && !s.live) return;
  if (MODE != kMixed || s.fast) {
    float x[8], y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float na = j & 1 ? b[j >> 1] : a[j >> 1], nb = j & 1 ? b[4 + (j >> 1)] : a[4 + (j >> 1)];
      const bool split = MODE == kHalves || (MODE >= kMixed && s.split);
      x[j] = split ? a[j] : na;
      y[j] = split ? b[j] : nb;
    }
    if (P.past) {
      store8_full<true>(row + s.off[0], x);
      store8_full<true>(row + s.off[1], y);
    } else {
      store8_full<false>(row + s.off[0], x);
      store8_full<false>(row + s.off[1], y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int da = channel(P, s.p0 + j, 0), db = channel(P, s.p0 + j, 1);
      if (da < P.D) row[da] = from_f32<T>(a[j]);
      if (db < P.D) row[db] = from_f32<T>(b[j]);
    }
  }
}

// The sum over a row's lanes, in every one of them.
__device__ __forceinline__ float row_sum(float v, int lanes) {
  if (lanes >= 2) v = v + dpp_mov<DPP_XOR1>(v);
  if (lanes >= 4) v = v + dpp_mov<DPP_XOR2>(v);
  if (lanes >= 8) v = v + dpp_mov<DPP_HALF_MIRROR>(v);
  if (lanes >= 16) v = v + dpp_mov<DPP_MIRROR>(v);
  if (lanes >= 32) {
    const Halves h = halves16(v);
    v = h.a + h.b;
  }
  if (lanes >= 64) {
    const Halves h = halves32(v);
    v = h.a + h.b;
  }
  return v;
}

// Two floats per pair: a weight of either side, or cos and sin.
struct Two {
  float a, b;
};
// The weights of queries and keys in pair order, ones where there are none; padded to
// the pairs of all lanes, as the turns are.
__device__ __forceinline__ void form_weights(Two* w, const QkPlan& P, const float* w_q, const float* w_k) {
  const int n = 8 * P.lanes;
  for (int i = threadIdx.x; i < 2 * n; i += kThreads) {
    const float* p = i < n ? w_q : w_k;
    const int da = channel(P, i < n ? i : i - n, 0), db = channel(P, i < n ? i : i - n, 1);
    w[i] = {p && da < P.D ? p[da] : 1.0f, p && db < P.D ? p[db] : 1.0f};
  }
}

// cos and sin of pos * f, both with all their digits: the turns pos f / 2 pi as two
// float64 words (the product of 31 and 24 bits, and that with a two-word 1 / 2 pi), less
// the nearest quarter turn, so that what float32 takes over is small where the sine or
// cosine is.
__device__ __forceinline__ Two cos_sin(int32_t pos, float f) {
  constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnLo = -0x1.6b01ec5417056p-57;
  const double p = static_cast<double>(pos), q = p * f, q_lo = fma(p, static_cast<double>(f), -q);
  const double x = q * kTurn, x_lo = fma(q, kTurn, -x) + fma(q_lo, kTurn, q * kTurnLo);
  const double k = rint(4.0 * x);
  Two u;
  float s, c;
  sincospif(static_cast<float>(2.0 * ((x - 0.25 * k) + x_lo)), &s, &c);
  const int quarter = static_cast<int>(static_cast<int64_t>(k) & 3);
  const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  u.a = quarter == 1 || quarter == 2 ? -a : a;
  u.b = quarter >= 2 ? -b : b;
  return u;
}

// cos and sin of every pair of the tokens [t0, t0 + n).
__device__ __forceinline__ void form_turns(Two* turns, const QkPlan& P, int64_t t0, int n) {
  const int log_n = 31 - __builtin_clz(8 * P.lanes);
  for (int i = threadIdx.x; i < n << log_n; i += kThreads) {
    const int t = i >> log_n, p = i & ((1 << log_n) - 1);
    Two u{1.0f, 0.0f};
    if (p < P.half) {
      const int ax = P.axis ? P.axis[p] : 0;
      if (ax >= 0 && ax < P.axes) u = cos_sin(P.pos[ax * P.pos_ld + t0 + t], P.inv_freq[p]);
    }
    turns[i] = u;
  }
}

__device__ __forceinline__ void turn_pairs(const Two* u, float way, float (&a)[8], float (&b)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = a[j], y = b[j], c = u[j].a, sn = way * u[j].b;
    a[j] = __builtin_fmaf(x, c, -(y * sn));
    b[j] = __builtin_fmaf(y, c, x * sn);
  }
}

template <typename T, int MODE>
__global__ __launch_bounds__(kThreads) void qk_norm_kernel(QkPlan P, Heads<const T> q, Heads<T> qo, int Hq,
                                                           const float* __restrict__ w_q, Heads<const T> k, Heads<T> ko,
                                                           int Hk, const float* __restrict__ w_k) {
  __shared__ __align__(16) Two turns[kTurns], weights[kMaxD];
  const Spot s = spot_of(P);
  const int group = threadIdx.x / P.lanes, row_pairs = 8 * P.lanes;
  form_weights(weights, P, w_q, w_k);
  __syncthreads();
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.tokens; t0 < P.T; t0 += static_cast<int64_t>(gridDim.x) * P.tokens) {
    const int n = P.T - t0 < P.tokens ? static_cast<int>(P.T - t0) : P.tokens;
    if (P.half) {
      __syncthreads();
      form_turns(turns, P, t0, n);
      __syncthreads();
    }
    for (int side = 0; side < 2; ++side) {
      const Heads<const T>& in = side ? k : q;
      const Heads<T>& out = side ? ko : qo;
      const int H = side ? Hk : Hq;
      if (H == 0) continue;
      const Two* w = weights + side * row_pairs + s.p0;
      for (int i = group; i < n * H; i += P.groups) {
        const int t = i / H, h = i - t * H;
        Row<T, MODE> row;
        float a[8], b[8];
        row.load(in.row(t0 + t, h), P, s);
        row.get(P, s, a, b);
        if (P.norm != DET_NORM_NONE) {
          float m = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) m = __builtin_fmaf(a[j], a[j], __builtin_fmaf(b[j], b[j], m));
          const float r = 1.0f / sqrtf(__builtin_fmaf(row_sum(m, P.lanes), P.inv, P.eps));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            a[j] *= r;
            b[j] *= r;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j] *= w[j].a;
          b[j] *= w[j].b;
        }
        if (s.p0 < P.half) turn_pairs(turns + t * row_pairs + s.p0, 1.0f, a, b);
        put_row<MODE>(out.row(t0 + t, h), P, s, a, b);
      }
    }
  }
}

template <typename T, int MODE>
__global__ __launch_bounds__(kThreads, MODE == kMixed ? 2 : 4) void qk_norm_bwd_kernel(QkPlan P, Heads<const T> dyq, Heads<const T> q, Heads<T> dq,
                                                               int Hq, const float* __restrict__ w_q, Heads<const T> dyk,
                                                               Heads<const T> k, Heads<T> dk, int Hk,
                                                               const float* __restrict__ w_k, float* __restrict__ slots) {
  __shared__ __align__(16) Two turns[kTurns], weights[kMaxD];
  __shared__ float part[kThreads / 64][kMaxD];
  const Spot s = spot_of(P);
  const int group = threadIdx.x / P.lanes, row_pairs = 8 * P.lanes;
  form_weights(weights, P, w_q, w_k);
  __syncthreads();
  float sa[2][8] = {}, sb[2][8] = {};
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.tokens; t0 < P.T; t0 += static_cast<int64_t>(gridDim.x) * P.tokens) {
    const int n = P.T - t0 < P.tokens ? static_cast<int>(P.T - t0) : P.tokens;
    if (P.half) {
      __syncthreads();
      form_turns(turns, P, t0, n);
      __syncthreads();
    }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const Heads<const T>&in = side ? k : q, &dy = side ? dyk : dyq;
      const Heads<T>& out = side ? dk : dq;
      const int H = side ? Hk : Hq;
      if (H == 0) continue;
      const Two* w = weights + side * row_pairs + s.p0;
      for (int i = group; i < n * H; i += P.groups) {
        const int t = i / H, h = i - t * H;
        Row<T, MODE> rx, rd;
        float a[8], b[8], da[8], db[8];
        rx.load(in.row(t0 + t, h), P, s);
        rd.load(dy.row(t0 + t, h), P, s);
        rx.get(P, s, a, b);
        rd.get(P, s, da, db);
        if (s.p0 < P.half) turn_pairs(turns + t * row_pairs + s.p0, -1.0f, da, db);
        float r = 1.0f;
        if (P.norm != DET_NORM_NONE) {
          float m = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) m = __builtin_fmaf(a[j], a[j], __builtin_fmaf(b[j], b[j], m));
          r = 1.0f / sqrtf(__builtin_fmaf(row_sum(m, P.lanes), P.inv, P.eps));
        }
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j] *= r;
          b[j] *= r;
          sa[side][j] = __builtin_fmaf(da[j], a[j], sa[side][j]);
          sb[side][j] = __builtin_fmaf(db[j], b[j], sb[side][j]);
          da[j] *= w[j].a;
          db[j] *= w[j].b;
          m = __builtin_fmaf(da[j], a[j], __builtin_fmaf(db[j], b[j], m));
        }
        if (P.norm != DET_NORM_NONE) {
          m = row_sum(m, P.lanes) * P.inv;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            da[j] = r * __builtin_fmaf(-a[j], m, da[j]);
            db[j] = r * __builtin_fmaf(-b[j], m, db[j]);
          }
        }
        put_row<MODE>(out.row(t0 + t, h), P, s, da, db);
      }
    }
  }
  if (!slots) return;
  // the rows side by side in a wave, then the waves; slot [workgroup][side][D]
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float a = sa[side][j], b = sb[side][j];
      for (int d = P.lanes; d < 64; d <<= 1) {
        a += __shfl_xor(a, d);
        b += __shfl_xor(b, d);
      }
      const int ca = channel(P, s.p0 + j, 0), cb = channel(P, s.p0 + j, 1);
      if (static_cast<int>(threadIdx.x & 63) < P.lanes) {
        if (ca < P.D) part[threadIdx.x >> 6][ca] = a;
        if (cb < P.D) part[threadIdx.x >> 6][cb] = b;
      }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < P.D; d += kThreads) {
      float t = part[0][d];
#pragma unroll
      for (int w = 1; w < kThreads / 64; ++w) t += part[w][d];
      slots[(static_cast<int64_t>(blockIdx.x) * 2 + side) * P.D + d] = t;
    }
  }
}

// Workgroup (x, side): 64 channels of one parameter; wave w adds the slots w, w + 16, ...
__global__ __launch_bounds__(64 * kFoldWaves) void qk_norm_fold_kernel(const float* __restrict__ slots, int n, int D,
                                                                       float* __restrict__ dw_q, float* __restrict__ dw_k) {
  __shared__ double part[kFoldWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, side = blockIdx.y, d = blockIdx.x * 64 + lane;
  float* dw = side ? dw_k : dw_q;
  if (!dw) return;
  const float* p = slots + static_cast<int64_t>(side) * D + (d < D ? d : 0);
  double t = 0.0;
#pragma unroll 8
  for (int i = wave; i < n; i += kFoldWaves) t += p[static_cast<int64_t>(i) * 2 * D];
  part[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && d < D) {
    t = part[0][lane];
#pragma unroll
    for (int w = 1; w < kFoldWaves; ++w) t += part[w][lane];
    dw[d] += static_cast<float>(t);
  }
}

int lanes_for(int64_t D) {
  int l = 1;
  while (16 * l < D) l *= 2;
  return l;
}
// Workgroups: as many as are at work at once (the backward leaves a slot for each).
int64_t most_groups(bool bwd) { return bwd ? 1024 : 4096; }
// Tokens of a workgroup's turn: one round of its lanes at least while every compute unit has a
// workgroup, up to four while there are 1024, and the same number of turns for all; their
// sines have to fit. (8191 tokens of 18 heads, backward: one turn of 8 tokens for each of 1024
// workgroups, all at work at once, 30 us; 1171 turns of 7 tokens, three workgroups to a compute
// unit, 39 us.)
int64_t tokens_for(int64_t T, int64_t D, int64_t heads, bool bwd) {
  const int64_t rows = kThreads / lanes_for(D), room = kTurns / (8 * lanes_for(D));
  const auto lower = [](int64_t a, int64_t b) { return a < b ? a : b; };
  int64_t n = lower(ceil_div(4 * rows, heads), ceil_div(T, 1024));
  const int64_t one = lower(rows / heads, T / 256);
  n = lower(n > one ? n : one, room);
  if (n < 1) n = 1;
  const int64_t turns = ceil_div(ceil_div(T, n), most_groups(bwd));
  return turns > 1 ? lower(n, ceil_div(T, most_groups(bwd) * turns)) : n;
}
int64_t groups_for(int64_t T, int64_t tokens, bool bwd) {
  const int64_t n = ceil_div(T, tokens);
  return n < most_groups(bwd) ? n : most_groups(bwd);
}
size_t ws_bytes_for(int64_t T, int64_t D, int64_t heads) {
  return T == 0 || D == 0 || heads == 0
             ? 0
             : DET_WS_HEADER_BYTES +
                   align_up(static_cast<size_t>(groups_for(T, tokens_for(T, D, heads, true), true) * 2 * D) * 4, 256);
}

int check_sizes(const char* what, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R) {
  if (T < 0 || D < 0 || Hq < 0 || Hk < 0) return set_error(DET_ERR_INVALID_ARG, "%s: sizes must be >= 0", what);
  if (R < 0 || R > D || R % 2)
    return set_error(DET_ERR_INVALID_ARG, "%s: the rotated channels must be even and at most D, got %lld", what, (long long)R);
  if (D > kMaxD) return set_error(DET_ERR_UNSUPPORTED, "%s: D must be <= %d, got %lld", what, kMaxD, (long long)D);
  if (Hq > 65535 || Hk > 65535 || T > (int64_t(1) << 40)) return set_error(DET_ERR_UNSUPPORTED, "%s: problem too large", what);
  return DET_OK;
}

// The checks that both directions share, and the plan.
int make_plan(const char* what, int dtype, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int norm, double eps, const int32_t* pos,
              int64_t pos_ld, int64_t axes, const float* inv_freq, const int32_t* axis, int64_t R, int pairs, bool bwd, QkPlan& P) {
  if (int s = check_float_dtype(what, dtype)) return s;
  if (norm != DET_NORM_NONE && norm != DET_NORM_RMS && norm != DET_NORM_L2)
    return set_error(DET_ERR_INVALID_ARG, "%s: unknown norm %d", what, norm);
  if (pairs != DET_PAIRS_HALVES && pairs != DET_PAIRS_NEIGHBOURS)
    return set_error(DET_ERR_INVALID_ARG, "%s: unknown pairs %d", what, pairs);
  if (!(eps >= 0.0 && eps < 1e30)) return set_error(DET_ERR_INVALID_ARG, "%s: eps must be >= 0 and finite", what);
  if (R > 0 && T > 0 && Hq + Hk > 0) {
    if (!pos || !inv_freq) return set_error(DET_ERR_INVALID_ARG, "%s: a rotation needs pos and inv_freq", what);
    if (axes < 1 || axes > 65535) return set_error(DET_ERR_INVALID_ARG, "%s: axes must lie in [1, 65535]", what);
    if (axes > 1 && !axis) return set_error(DET_ERR_INVALID_ARG, "%s: several axes need the axis of every pair", what);
    if (axes > 1 && pos_ld < T) return set_error(DET_ERR_INVALID_ARG, "%s: row stride of pos < T", what);
    if (axes > 1 && pos_ld > (int64_t(1) << 44) / axes) return set_error(DET_ERR_UNSUPPORTED, "%s: pos is too large", what);
  }
  const int lanes = lanes_for(D);
  P = QkPlan{T, (int)D, (int)(R / 2), lanes, (int)tokens_for(T, D, Hq + Hk > 0 ? Hq + Hk : 1, bwd), kThreads / lanes, norm,
             pairs == DET_PAIRS_HALVES, past_caches(T * (Hq + Hk) * D * static_cast<int64_t>(dtype_size(dtype))),
             static_cast<float>(eps), norm == DET_NORM_RMS ? static_cast<float>(1.0 / (D > 0 ? D : 1)) : 1.0f,
             pos, axis, axes > 1 ? pos_ld : 0, (int)axes, inv_freq};
  return DET_OK;
}
// Whether every lane of a row owns whole runs, if any, and all of one kind. (40 heads of 128 channels, 64 of
// them turned in halves, 16384 tokens, forward: 67 us; 60 of them, by elements: 141 us.)
int mode_of(const QkPlan& P) {
  if (P.D % 16) return kMixed;
  if (P.halves && P.half) return 2 * P.half == P.D ? kHalves : P.half % 8 == 0 ? kEither : kMixed;
  return kNeighbours;
}

}  // namespace
}  // namespace detgrad

using namespace detgrad;

#define DET_QK_LAUNCH(KERNEL, T, ...)                                                                       \
  switch (mode_of(P)) {                                                                                     \
    case kHalves: hipLaunchKernelGGL((KERNEL<T, kHalves>), grid, dim3(kThreads), 0, st, __VA_ARGS__); break; \
    case kNeighbours:                                                                                       \
      hipLaunchKernelGGL((KERNEL<T, kNeighbours>), grid, dim3(kThreads), 0, st, __VA_ARGS__);               \
      break;                                                                                                \
    case kEither: hipLaunchKernelGGL((KERNEL<T, kEither>), grid, dim3(kThreads), 0, st, __VA_ARGS__); break; \
    default: hipLaunchKernelGGL((KERNEL<T, kMixed>), grid, dim3(kThreads), 0, st, __VA_ARGS__);             \
  }

extern "C" int det_qk_norm(const void* q, int64_t q_st, int64_t q_sh, int64_t Hq, const void* k, int64_t k_st, int64_t k_sh,
                           int64_t Hk, int dtype, int64_t T, int64_t D, const float* w_q, const float* w_k, int norm,
                           double eps, const int32_t* pos, int64_t pos_ld, int64_t axes, const float* inv_freq,
                           const int32_t* axis, int64_t R, int pairs, void* q_out, int64_t qo_st, int64_t qo_sh,
                           void* k_out, int64_t ko_st, int64_t ko_sh, void* stream) {
  const char* what = "qk_norm";
  if (int s = check_sizes(what, T, Hq, Hk, D, R)) return s;
  QkPlan P;
  if (int s = make_plan(what, dtype, T, Hq, Hk, D, norm, eps, pos, pos_ld, axes, inv_freq, axis, R, pairs, false, P)) return s;
  if (T == 0 || D == 0 || Hq + Hk == 0) return ok();
  if ((Hq && (!q || !q_out)) || (Hk && (!k || !k_out))) return set_error(DET_ERR_INVALID_ARG, "%s: NULL pointer", what);
  const size_t es = dtype_size(dtype);
  Buf b[4];
  if (int s = delta_buf(what, "q_out", q_out, T, Hq, D, qo_st, qo_sh, es, b[0])) return s;
  if (int s = delta_buf(what, "k_out", k_out, T, Hk, D, ko_st, ko_sh, es, b[1])) return s;
  if (int s = delta_buf(what, "q", q, T, Hq, D, q_st, q_sh, es, b[2])) return s;
  if (int s = delta_buf(what, "k", k, T, Hk, D, k_st, k_sh, es, b[3])) return s;
  const Buf ins[] = {b[2], b[3], {"w_q", range1d(w_q, D * 4)}, {"w_k", range1d(w_k, D * 4)},
                     {"pos", range1d(R ? pos : nullptr, ((axes > 1 ? (axes - 1) * pos_ld : 0) + T) * 4)},
                     {"inv_freq", range1d(R ? inv_freq : nullptr, R * 2)}, {"axis", range1d(R ? axis : nullptr, R * 2)}};
  if (int s = check_buffers(what, b, 2, ins, 7)) return s;
  const dim3 grid(static_cast<uint32_t>(groups_for(T, P.tokens, false)));
  const hipStream_t st = as_stream(stream);
#define DET_QK_FWD(E)                                                                                                  \
  DET_QK_LAUNCH(qk_norm_kernel, E, P, Heads<const E>{static_cast<const E*>(q), q_st, q_sh},                            \
                Heads<E>{static_cast<E*>(q_out), qo_st, qo_sh}, (int)Hq, w_q,                                          \
                Heads<const E>{static_cast<const E*>(k), k_st, k_sh}, Heads<E>{static_cast<E*>(k_out), ko_st, ko_sh},  \
                (int)Hk, w_k)
  if (dtype == DET_BF16) {
    DET_QK_FWD(uint16_t)
  } else {
    DET_QK_FWD(float)
  }
#undef DET_QK_FWD
  return check_launch("det_qk_norm");
}

extern "C" int det_qk_norm_bwd_workspace_size(int64_t T, int64_t Hq, int64_t Hk, int64_t D, size_t* bytes) {
  if (!bytes) return set_error(DET_ERR_INVALID_ARG, "qk_norm_bwd: bytes is NULL");
  if (int s = check_sizes("qk_norm_bwd", T, Hq, Hk, D, 0)) return s;
  *bytes = ws_bytes_for(T, D, Hq + Hk);
  return ok();
}

extern "C" int det_qk_norm_bwd(const void* dq_out, int64_t dqo_st, int64_t dqo_sh, const void* dk_out, int64_t dko_st,
                               int64_t dko_sh, const void* q, int64_t q_st, int64_t q_sh, int64_t Hq, const void* k,
                               int64_t k_st, int64_t k_sh, int64_t Hk, int dtype, int64_t T, int64_t D, const float* w_q,
                               const float* w_k, int norm, double eps, const int32_t* pos, int64_t pos_ld, int64_t axes,
                               const float* inv_freq, const int32_t* axis, int64_t R, int pairs, void* dq, int64_t dq_st,
                               int64_t dq_sh, void* dk, int64_t dk_st, int64_t dk_sh, float* dw_q, float* dw_k, void* ws,
                               size_t ws_bytes, void* stream) {
  const char* what = "qk_norm_bwd";
  if (int s = check_sizes(what, T, Hq, Hk, D, R)) return s;
  QkPlan P;
  if (int s = make_plan(what, dtype, T, Hq, Hk, D, norm, eps, pos, pos_ld, axes, inv_freq, axis, R, pairs, true, P)) return s;
  if ((w_q != nullptr) != (dw_q != nullptr) || (w_k != nullptr) != (dw_k != nullptr))
    return set_error(DET_ERR_INVALID_ARG, "%s: w_q goes with dw_q, w_k with dw_k", what);
  if (T == 0 || D == 0 || Hq + Hk == 0) return ok();
  if ((Hq && (!q || !dq_out || !dq)) || (Hk && (!k || !dk_out || !dk)))
    return set_error(DET_ERR_INVALID_ARG, "%s: NULL pointer", what);
  const size_t es = dtype_size(dtype);
  Buf b[6];
  if (int s = delta_buf(what, "dq", dq, T, Hq, D, dq_st, dq_sh, es, b[0])) return s;
  if (int s = delta_buf(what, "dk", dk, T, Hk, D, dk_st, dk_sh, es, b[1])) return s;
  if (int s = delta_buf(what, "q", q, T, Hq, D, q_st, q_sh, es, b[2])) return s;
  if (int s = delta_buf(what, "k", k, T, Hk, D, k_st, k_sh, es, b[3])) return s;
  if (int s = delta_buf(what, "dq_out", dq_out, T, Hq, D, dqo_st, dqo_sh, es, b[4])) return s;
  if (int s = delta_buf(what, "dk_out", dk_out, T, Hk, D, dko_st, dko_sh, es, b[5])) return s;
  const size_t need = w_q || w_k ? ws_bytes_for(T, D, Hq + Hk) : 0;
  if (int s = check_workspace(ws, ws_bytes, need)) return s;
  const Buf outs[] = {b[0], b[1], {"dw_q", range1d(dw_q, D * 4)}, {"dw_k", range1d(dw_k, D * 4)},
                      {"the workspace", range1d(need ? ws : nullptr, ws_bytes)}};
  const Buf ins[] = {b[2], b[3], b[4], b[5], {"w_q", range1d(w_q, D * 4)}, {"w_k", range1d(w_k, D * 4)},
                     {"pos", range1d(R ? pos : nullptr, ((axes > 1 ? (axes - 1) * pos_ld : 0) + T) * 4)},
                     {"inv_freq", range1d(R ? inv_freq : nullptr, R * 2)}, {"axis", range1d(R ? axis : nullptr, R * 2)}};
  if (int s = check_buffers(what, outs, 5, ins, 9)) return s;
  const int64_t groups = groups_for(T, P.tokens, true);
  const dim3 grid(static_cast<uint32_t>(groups));
  const hipStream_t st = as_stream(stream);
  auto* slots = need ? reinterpret_cast<float*>(static_cast<char*>(ws) + DET_WS_HEADER_BYTES) : nullptr;
#define DET_QK_BWD(E)                                                                                                 \
  DET_QK_LAUNCH(qk_norm_bwd_kernel, E, P, Heads<const E>{static_cast<const E*>(dq_out), dqo_st, dqo_sh},              \
                Heads<const E>{static_cast<const E*>(q), q_st, q_sh}, Heads<E>{static_cast<E*>(dq), dq_st, dq_sh},    \
                (int)Hq, w_q, Heads<const E>{static_cast<const E*>(dk_out), dko_st, dko_sh},                          \
                Heads<const E>{static_cast<const E*>(k), k_st, k_sh}, Heads<E>{static_cast<E*>(dk), dk_st, dk_sh},    \
                (int)Hk, w_k, slots)
  if (dtype == DET_BF16) {
    DET_QK_BWD(uint16_t)
  } else {
    DET_QK_BWD(float)
  }
#undef DET_QK_BWD
  if (need)
    hipLaunchKernelGGL(qk_norm_fold_kernel, dim3(static_cast<uint32_t>(ceil_div(D, 64)), 2), dim3(64 * kFoldWaves), 0, st,
                       slots, static_cast<int>(groups), (int)D, dw_q, dw_k);
  return check_launch("det_qk_norm_bwd");
}
