// det_block_norm / det_block_norm_bwd: the boundary between two residual blocks
// in one pass: the norm after the first block with its gate and residual scale,
// the residual sum, and the norm before the second.
//
//   n = f rstd_f w_post,  rstd_f = 1 / sqrt(mean(f^2) + eps)      (w_post NULL: n = f)
//   y = x + alpha s n,    s = sigmoid(gate)                        (alpha, gate NULL: factors of 1)
//   h = y rstd_y w_pre,   rstd_y = 1 / sqrt(mean(y^2) + eps)      (w_pre NULL: no h)
//
// y enters its norm before it is rounded to the output type, and the backward
// recomputes it in float32 from x and f, so it needs no copy of y.
//
//   yh = y rstd_y, u = w_pre dh:  D = dy + rstd_y (u - yh mean(u yh))   (w_pre NULL: D = dy)
//   dx = D;  dw_pre += sum dh yh
//   dn = D alpha s:  dgate = dn n (1 - s)  (its row sum for a gate per token)
//   fh = f rstd_f:   df = rstd_f (w_post dn - fh mean(w_post dn fh))   (w_post NULL: df = dn)
//   A = sum D s fh over the tokens:  dw_post += alpha A,  dalpha += w_post A  (one column sum for both)
//
// A workgroup owns whole rows, eight (or sixteen) consecutive channels per
// thread, so a row's sums are a wave tree and one exchange through LDS, and the
// parameters and the parameter gradients' running sums of a thread's channels
// stay in registers while it walks its rows. The parameter gradients are column
// sums: workgroup b adds rows b, b + G, b + 2G, ... in order into its own slot
// (no atomics), a fold adds the slots in a fixed order in float64, and once into the output.
//
// Both directions are bound by the [T, D] tensors: five read or written forward
// (8192 x 4096 bf16, a gate per channel: 67 us, 5.0 TB/s), eight backward (16384 x
// 8192 bf16: 391 us, 5.5 TB/s, and 6.5 for the fold).
#include "rowops.hpp"

namespace detgrad {
namespace {

constexpr int kMaxD = 16384;

// Sum of v over the workgroup, in every thread: each wave's tree, then the waves
// left to right. `buf` has one float per wave; two buffers used in turn need no
// barrier between the reads of one and the writes of the next.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* buf) {
  v = lanes_sum<64>(v);
  if constexpr (THREADS == 64) {
    return v;
  } else {
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = buf[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) s += buf[w];
    return s;
  }
}

// 1 / (1 + 2^(-g log2 e)) by the hardware's exponential and reciprocal: within
// (|g| + 3) units in the last place of a float32 sigmoid.
__device__ __forceinline__ float sigmoid_f(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * kLog2e));
}

// The backward needs s = sigmoid(g) and 1 - s with all their digits (1 - s formed
// from a rounded s has lost 1e-4 of its value at g = 9 and all of it from g = 17
// on), in one register: the smaller of the two, t / (1 + t) with t = exp(-|g|), with
// g's sign. The other is 1 less it.
__device__ __forceinline__ float gate_code(float g) {
  const float t = __builtin_amdgcn_exp2f(-fabsf(g) * kLog2e);
  return copysignf(t * __builtin_amdgcn_rcpf(1.0f + t), g);
}
__device__ __forceinline__ float gate_open(float w) { return __float_as_int(w) < 0 ? -w : 1.0f - w; }
__device__ __forceinline__ float gate_shut(float w) { return __float_as_int(w) < 0 ? 1.0f + w : w; }

enum GateKind { kGateNone = 0, kGateRow = 1, kGateFull = 2 };

struct NormParams {
  const float *w_post, *alpha, *w_pre;  // [D] float32, NULL: not applied
  float eps, inv_d;
  int64_t rows, D;
};

// Rows of fewer than eight channels only reach the 64-thread instances.
template <bool TINY>
__device__ __forceinline__ void load_param(const float* p, const Cols<TINY>& c, float (&v)[8]) {
  if (p) {
    Raw8<float> r;
    load_cols(r, p, c);
    get_cols(r, c, 0.0f, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 1.0f;
  }
}

template <typename T, int THREADS, int NV, bool PAST>
__global__ __launch_bounds__(THREADS) void norm_fwd_kernel(const T* __restrict__ x, int64_t ld_x,
                                                           const T* __restrict__ f, int64_t ld_f,
                                                           const T* __restrict__ gate, int64_t ld_g, int gate_kind,
                                                           NormParams P, T* __restrict__ y, int64_t ld_y,
                                                           T* __restrict__ h, int64_t ld_h,
                                                           float* __restrict__ rstd_post,
                                                           float* __restrict__ rstd_pre) {
  __shared__ float buf[2][THREADS / 64];
  const bool post = P.w_post != nullptr, pre = P.w_pre != nullptr;
  float wp[NV][8], wq[NV][8];  // w_post alpha, w_pre
  Cols<THREADS == 64> c[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    c[i].set((i * THREADS + threadIdx.x) * 8, static_cast<int>(P.D), THREADS * NV * 8);
    float al[8];
    load_param(P.w_post, c[i], wp[i]);
    load_param(P.alpha, c[i], al);
    load_param(P.w_pre, c[i], wq[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) wp[i][j] *= al[j];
  }
  for (int64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
    float xv[NV][8], fv[NV][8], gv[NV][8];
    {
      Raw8<T> rx[NV], rf[NV], rg[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        load_cols(rf[i], f + r * ld_f, c[i]);
        load_cols(rx[i], x + r * ld_x, c[i]);
        if (gate_kind == kGateFull) load_cols(rg[i], gate + r * ld_g, c[i]);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        get_cols(rf[i], c[i], 0.0f, fv[i]);
        get_cols(rx[i], c[i], 0.0f, xv[i]);
        if (gate_kind == kGateFull) rg[i].get(gv[i]);
      }
    }
    const float s_row = gate_kind == kGateRow ? sigmoid_f(to_f32(gate[r * ld_g])) : 1.0f;
    float rp = 1.0f;
    if (post) {
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) q += fv[i][j] * fv[i][j];
      rp = 1.0f / sqrtf(block_sum<THREADS>(q, buf[0]) * P.inv_d + P.eps);
      if (threadIdx.x == 0) rstd_post[r] = rp;
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float s = gate_kind == kGateFull ? sigmoid_f(gv[i][j]) : s_row;
        xv[i][j] += fv[i][j] * rp * wp[i][j] * s;
        q += xv[i][j] * xv[i][j];
      }
      store_cols<PAST>(y + r * ld_y, c[i], xv[i]);
    }
    if (pre) {
      const float rq = 1.0f / sqrtf(block_sum<THREADS>(q, buf[1]) * P.inv_d + P.eps);
      if (threadIdx.x == 0) rstd_pre[r] = rq;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) xv[i][j] = xv[i][j] * rq * wq[i][j];
        store_cols<PAST>(h + r * ld_h, c[i], xv[i]);
      }
    }
    // with one sum per row the same buffer serves every row
    if (THREADS > 64 && post != pre) __syncthreads();
  }
}

// One row of the backward's inputs as loaded.
template <typename T, int NV>
struct BwdRow {
  Raw8<T> f[NV], g[NV], x[NV], u[NV], d[NV];
  float rp, rq, g_row;
};

template <typename T>
struct BwdIn {
  const T *dy, *dh, *x, *f, *gate;
  int64_t ld_dy, ld_dh, ld_x, ld_f, ld_g;
  const float *rstd_post, *rstd_pre;
  bool row_gate;  // one gate per token
};

// Calls whose outputs pass the caches wait for f before the other tensors are asked
// for: fewer streams of memory open at once (8192 x 4096 float32: 224 us against
// 239, 16384 x 8192 bf16: 397 against 401; smaller calls lose 2 us at 3001 x 1407).
template <bool FULL, bool PAST, typename T, int NV, bool TINY>
__device__ __forceinline__ void load_row(BwdRow<T, NV>& R, const BwdIn<T>& I, bool post, bool pre, int64_t r,
                                         const Cols<TINY> (&c)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_cols(R.f[i], I.f + r * I.ld_f, c[i]);
    if constexpr (PAST) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (FULL) load_cols(R.g[i], I.gate + r * I.ld_g, c[i]);
    if (pre) {
      load_cols(R.x[i], I.x + r * I.ld_x, c[i]);
      load_cols(R.u[i], I.dh + r * I.ld_dh, c[i]);
    }
    load_cols(R.d[i], I.dy + r * I.ld_dy, c[i]);
  }
  R.rp = post ? I.rstd_post[r] : 1.0f;
  R.rq = pre ? I.rstd_pre[r] : 1.0f;
  R.g_row = I.row_gate ? to_f32(I.gate[r * I.ld_g]) : 0.0f;
}

// A workgroup's slot holds A and dw_pre. The next row's loads are issued as soon
// as the current row is unpacked (bf16; a float32 row would take twice the
// registers). The parameters of a thread's channels sit in LDS (each thread
// reads back what it wrote, 16 bytes per lane side by side), which leaves the
// registers to the running sums, two rows and four waves per SIMD. FULL: a gate
// per channel (else one per token or none, and no register holds one). For D > 8192
// a thread has 16 channels: their running sums take the LDS instead, the
// parameters are read again for every row, and part of the row still spills
// (4096 x 16384 bf16: 381 us, 2.8 TB/s, against 5.5 at 16384 x 8192).
template <typename T, int THREADS, int NV, bool PAST, bool FULL>
__global__ __launch_bounds__(THREADS, 4) void norm_bwd_kernel(BwdIn<T> I, NormParams P, T* __restrict__ dx,
                                                              int64_t ld_dx, T* __restrict__ df, int64_t ld_df,
                                                              T* __restrict__ dgate, int64_t ld_dg,
                                                              float* __restrict__ slots) {
  constexpr bool kWide = NV > 1, kAhead = !kWide && sizeof(T) == 2;
  constexpr int kKept = 2 * NV;  // LDS: per thread, kKept sets of eight floats
  __shared__ float buf[2][THREADS / 64];
  __shared__ f32x4 kept[kKept][2][THREADS];
  const bool post = P.w_post != nullptr, pre = P.w_pre != nullptr;
  const bool second = post || I.row_gate;  // a second sum over the row is needed
  const auto put = [&](int k, const float(&w)[8]) {
    kept[k][0][threadIdx.x] = f32x4{w[0], w[1], w[2], w[3]};
    kept[k][1][threadIdx.x] = f32x4{w[4], w[5], w[6], w[7]};
  };
  const auto get = [&](int k, float(&w)[8]) {
    const f32x4 a = kept[k][0][threadIdx.x], b = kept[k][1][threadIdx.x];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = a[j];
      w[4 + j] = b[j];
    }
  };
  float sum_a[NV][8] = {}, sum_pre[NV][8] = {};  // (wide: in LDS)
  Cols<THREADS == 64> c[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    c[i].set((i * THREADS + threadIdx.x) * 8, static_cast<int>(P.D), THREADS * NV * 8);
    if constexpr (kWide) {
      put(2 * i, sum_a[i]);
      put(2 * i + 1, sum_pre[i]);
    }
  }
  // parameters of piece i: 0 = w_post alpha, 1 = w_pre
  const auto load_params = [&](int k, int i, float(&w)[8]) {
    load_param(k == 0 ? P.w_post : P.w_pre, c[i], w);
    if (k == 0) {
      float al[8];
      load_param(P.alpha, c[i], al);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] *= al[j];
    }
  };
  if constexpr (!kWide) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float w[8];
      load_params(k, 0, w);
      put(k, w);
    }
  }
  const auto param = [&](int k, int i, float(&w)[8]) {
    if constexpr (kWide)
      load_params(k, i, w);
    else
      get(k, w);
  };
  // sum[j] += a[j] * b[j] for the columns of piece i
  const auto accumulate = [&](int which, int i, float(&sum)[8], const float(&a)[8], const float(&b)[8]) {
    float t[8];
    if constexpr (kWide) get(2 * i + which, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (kWide)
        t[j] = __builtin_fmaf(a[j], b[j], t[j]);
      else
        sum[j] = __builtin_fmaf(a[j], b[j], sum[j]);
    }
    if constexpr (kWide) put(2 * i + which, t);
  };
  BwdRow<T, NV> R;
  if constexpr (kAhead) load_row<FULL, PAST>(R, I, post, pre, blockIdx.x, c);  // the grid has at most `rows` workgroups
#pragma unroll 1
  for (int64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
    float d[NV][8], fh[NV][8], g[NV][8], yh[NV][8], u[NV][8];
    if constexpr (!kAhead) load_row<FULL, PAST>(R, I, post, pre, r, c);
    const float rp = R.rp, rq = R.rq;
    const float w_row = I.row_gate ? gate_code(R.g_row) : 0.0f, s_row = gate_open(w_row);  // (no gate: 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      get_cols(R.f[i], c[i], 0.0f, fh[i]);
      if (FULL) R.g[i].get(g[i]);
      if (pre) {
        get_cols(R.x[i], c[i], 0.0f, yh[i]);
        get_cols(R.u[i], c[i], 0.0f, u[i]);
      }
      get_cols(R.d[i], c[i], 0.0f, d[i]);
    }
    if constexpr (kAhead) {
      if (r + gridDim.x < P.rows) load_row<FULL, PAST>(R, I, post, pre, r + gridDim.x, c);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        fh[i][j] *= rp;
        if (FULL) g[i][j] = gate_code(g[i][j]);
      }
    if (pre) {
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float wp[8], wq[8];
        param(0, i, wp);
        param(1, i, wq);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          yh[i][j] = (yh[i][j] + fh[i][j] * wp[j] * (FULL ? gate_open(g[i][j]) : s_row)) * rq;
        accumulate(1, i, sum_pre[i], u[i], yh[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float w = u[i][j] * wq[j];
          q = __builtin_fmaf(w, yh[i][j], q);
          d[i][j] = __builtin_fmaf(rq, w, d[i][j]);
        }
      }
      const float m = rq * (block_sum<THREADS>(q, buf[0]) * P.inv_d);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) d[i][j] = __builtin_fmaf(-m, yh[i][j], d[i][j]);
    }
    // d = the gradient of y, u = w_post dn
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      store_cols<PAST>(dx + r * ld_dx, c[i], d[i]);
      float wp[8];
      param(0, i, wp);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (FULL) asm volatile("" : "+v"(g[i][j]));  // s is formed again, not kept since its first use (registers)
        d[i][j] *= FULL ? gate_open(g[i][j]) : s_row;
      }
      accumulate(0, i, sum_a[i], d[i], fh[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[i][j] = d[i][j] * wp[j];
        q = __builtin_fmaf(u[i][j], fh[i][j], q);
      }
      if constexpr (FULL) {
        float dg[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) dg[j] = u[i][j] * fh[i][j] * gate_shut(g[i][j]);
        store_cols<PAST>(dgate + r * ld_dg, c[i], dg);
      }
    }
    if (second) {
      const float tot = block_sum<THREADS>(q, buf[1]);
      if (I.row_gate && threadIdx.x == 0) dgate[r * ld_dg] = from_f32<T>(tot * gate_shut(w_row));
      if (post) {
        const float mean = tot * P.inv_d;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) u[i][j] = rp * __builtin_fmaf(-mean, fh[i][j], u[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) store_cols<PAST>(df + r * ld_df, c[i], u[i]);
    if (THREADS > 64 && second != pre) __syncthreads();
  }
  if (!slots) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float* o = slots + static_cast<int64_t>(blockIdx.x) * 2 * P.D;
    if constexpr (kWide) {
      get(2 * i, sum_a[i]);
      get(2 * i + 1, sum_pre[i]);
    }
    if (post || P.alpha) store_cols(o, c[i], sum_a[i]);
    if (pre) store_cols(o + P.D, c[i], sum_pre[i]);
  }
}

// Workgroup (64 columns, sum): wave w of 16 adds slots w, w + 16, ... in order in
// float64, the waves' sums meet left to right, the total (times its parameter) is
// rounded to float32 once and added into the output. Sixteen waves
// with 16 loads each in flight, since a call has few columns and the slots come
// from other XCDs' L2s.
struct NormGrads {
  float *w_post, *alpha, *w_pre;
};
constexpr int kFoldWaves = 16;
__global__ __launch_bounds__(64 * kFoldWaves) void norm_fold_kernel(const float* __restrict__ slots, int n_slots,
                                                                    NormParams P, NormGrads G) {
  __shared__ double part[kFoldWaves][64];
  const bool second = blockIdx.y == 1;  // dw_pre
  if (second ? !G.w_pre : !(G.w_post || G.alpha)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t D = P.D, col = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const float* p = slots + blockIdx.y * D + (col < D ? col : 0);
  double t = 0.0;
  for (int b = wave; b < n_slots; b += 16 * kFoldWaves) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = b + kFoldWaves * i;
      v[i] = p[static_cast<int64_t>(k < n_slots ? k : wave) * 2 * D];  // (a slot read already, and not added)
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) t += b + kFoldWaves * i < n_slots ? v[i] : 0.0f;
  }
  part[wave][lane] = t;
  __syncthreads();
  if (wave != 0 || col >= D) return;
  t = part[0][lane];
#pragma unroll
  for (int w = 1; w < kFoldWaves; ++w) t += part[w][lane];
  if (second) {
    G.w_pre[col] += static_cast<float>(t);
  } else {
    const double wp = P.w_post ? P.w_post[col] : 1.0f, al = P.alpha ? P.alpha[col] : 1.0f;
    if (G.w_post) G.w_post[col] += static_cast<float>(t * al);
    if (G.alpha) G.alpha[col] += static_cast<float>(t * wp);
  }
}

int threads_for(int64_t D) {
  int t = 64;
  while (t < 1024 && t * 8 < D) t *= 2;
  return t;
}

// Workgroups of a launch, from the shape alone. Enough to fill the compute units
// (forward: their 2048 threads twice over; backward: the 1024 threads its
// registers allow), but where the tokens are few, few enough that a workgroup
// walks three rows (forward: its parameters are loaded once) or six (backward:
// every workgroup also writes a slot of 8 bytes per channel, which the fold
// reads). Measured at 3001 x 1407 float32 (inputs in the caches): 16 + 21 + 5.5 us against
// 17 + 21.5 + 7.5 with all workgroups; at 8192 x 4096 bf16 (inputs in the caches) the forward
// takes 53 us with 2048 workgroups and 57 with 512.
int64_t groups_for(int64_t T, int64_t D, bool bwd) {
  const int64_t full = bwd ? 256 * (1024 / threads_for(D)) : 512 * (2048 / threads_for(D));
  const int64_t few = bwd ? 512 : 1024, rows = bwd ? 6 : 3;
  int64_t g = ceil_div(T, rows);
  if (g < few) g = few;
  if (g > full) g = full;
  return T < g ? T : g;
}
size_t ws_bytes_for(int64_t T, int64_t D) {
  return T == 0 || D == 0 ? 0
                          : DET_WS_HEADER_BYTES + align_up(static_cast<size_t>(groups_for(T, D, true) * 2 * D) * 4, 256);
}

int check_sizes(const char* what, int64_t T, int64_t D) {
  if (T < 0 || D < 0) return set_error(DET_ERR_INVALID_ARG, "%s: T and D must be >= 0", what);
  if (D > kMaxD) return set_error(DET_ERR_UNSUPPORTED, "%s: D must be <= %d, got %lld", what, kMaxD, (long long)D);
  if (T > (int64_t(1) << 40)) return set_error(DET_ERR_UNSUPPORTED, "%s: T must be <= 2^40", what);
  return DET_OK;
}
int check_ld(const char* what, const char* name, const void* p, int64_t ld, int64_t n, int64_t T) {
  if (!p) return DET_OK;
  if (ld < n) return set_error(DET_ERR_INVALID_ARG, "%s: row stride of %s < %lld", what, name, (long long)n);
  if (ld > (int64_t(1) << 44) / T) return set_error(DET_ERR_UNSUPPORTED, "%s: %s is too large", what, name);
  return DET_OK;
}

}  // namespace
}  // namespace detgrad

using namespace detgrad;

#define DET_NORM_FWD_KERNEL(T, THREADS, NV, ...)                                                                 \
  if (past)                                                                                                      \
    hipLaunchKernelGGL((norm_fwd_kernel<T, THREADS, NV, true>), grid, dim3(THREADS), 0, st, __VA_ARGS__);        \
  else                                                                                                           \
    hipLaunchKernelGGL((norm_fwd_kernel<T, THREADS, NV, false>), grid, dim3(THREADS), 0, st, __VA_ARGS__);       \
  break;
#define DET_NORM_BWD_KERNEL(T, THREADS, NV, ...)                                                                 \
  if (past && full)                                                                                              \
    hipLaunchKernelGGL((norm_bwd_kernel<T, THREADS, NV, true, true>), grid, dim3(THREADS), 0, st, __VA_ARGS__);  \
  else if (past)                                                                                                 \
    hipLaunchKernelGGL((norm_bwd_kernel<T, THREADS, NV, true, false>), grid, dim3(THREADS), 0, st, __VA_ARGS__); \
  else if (full)                                                                                                 \
    hipLaunchKernelGGL((norm_bwd_kernel<T, THREADS, NV, false, true>), grid, dim3(THREADS), 0, st, __VA_ARGS__); \
  else                                                                                                           \
    hipLaunchKernelGGL((norm_bwd_kernel<T, THREADS, NV, false, false>), grid, dim3(THREADS), 0, st, __VA_ARGS__); \
  break;
#define DET_NORM_LAUNCH(KERNEL, T, ...)        \
  switch (D > 8192 ? 2048 : threads_for(D)) {  \
    case 64: KERNEL(T, 64, 1, __VA_ARGS__)     \
    case 128: KERNEL(T, 128, 1, __VA_ARGS__)   \
    case 256: KERNEL(T, 256, 1, __VA_ARGS__)   \
    case 512: KERNEL(T, 512, 1, __VA_ARGS__)   \
    case 1024: KERNEL(T, 1024, 1, __VA_ARGS__) \
    default: KERNEL(T, 1024, 2, __VA_ARGS__)   \
  }

extern "C" int det_block_norm(const void* x, int64_t x_ld, const void* f, int64_t f_ld, const void* gate,
                              int64_t gate_ld, int64_t gate_cols, const float* w_post, const float* alpha,
                              const float* w_pre, int dtype, int64_t T, int64_t D, double eps, void* y, int64_t y_ld,
                              void* h, int64_t h_ld, float* rstd_post, float* rstd_pre, void* stream) {
  const char* what = "block_norm";
  if (int s = check_sizes(what, T, D)) return s;
  if (int s = check_float_dtype(what, dtype)) return s;
  if (!(eps >= 0.0 && eps < 1e30)) return set_error(DET_ERR_INVALID_ARG, "%s: eps must be >= 0 and finite", what);
  if (T == 0 || D == 0) return ok();
  if (!x || !f || !y) return set_error(DET_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if (gate && gate_cols != 1 && gate_cols != D)
    return set_error(DET_ERR_INVALID_ARG, "%s: gate_cols must be 1 or D, got %lld", what, (long long)gate_cols);
  if ((w_pre != nullptr) != (h != nullptr) || (w_pre != nullptr) != (rstd_pre != nullptr))
    return set_error(DET_ERR_INVALID_ARG, "%s: w_pre, h and rstd_pre go together", what);
  if ((w_post != nullptr) != (rstd_post != nullptr))
    return set_error(DET_ERR_INVALID_ARG, "%s: w_post and rstd_post go together", what);
  const struct {
    const char* name;
    const void* p;
    int64_t ld, cols;
  } rows[] = {{"x", x, x_ld, D}, {"f", f, f_ld, D}, {"gate", gate, gate_ld, gate_cols}, {"y", y, y_ld, D},
              {"h", h, h_ld, D}};
  Buf rr[5];
  for (int i = 0; i < 5; ++i) {
    if (int s = check_ld(what, rows[i].name, rows[i].p, rows[i].ld, rows[i].cols, T)) return s;
    rr[i] = buf_rows(rows[i].name, rows[i].p, T, rows[i].cols, rows[i].ld, dtype_size(dtype));
  }
  const Buf outs[] = {rr[3], rr[4],
                      {"rstd_post", range1d(rstd_post, T * 4)},
                      {"rstd_pre", range1d(rstd_pre, T * 4)}};
  const Buf ins[] = {rr[0], rr[1], rr[2],
                     {"w_post", range1d(w_post, D * 4)},
                     {"alpha", range1d(alpha, D * 4)},
                     {"w_pre", range1d(w_pre, D * 4)}};
  if (int s = check_buffers(what, outs, 4, ins, 6)) return s;
  const NormParams P{w_post, alpha, w_pre, static_cast<float>(eps), static_cast<float>(1.0 / D), T, D};
  const int kind = !gate ? kGateNone : (gate_cols == D ? kGateFull : kGateRow);
  const dim3 grid(static_cast<uint32_t>(groups_for(T, D, false)));
  const bool past = past_caches(T * D * static_cast<int64_t>(dtype_size(dtype)) * (h ? 2 : 1));
  const hipStream_t st = as_stream(stream);
#define DET_NORM_FWD(E)                                                                                             \
  DET_NORM_LAUNCH(DET_NORM_FWD_KERNEL, E, static_cast<const E*>(x), x_ld, static_cast<const E*>(f), f_ld,           \
                  static_cast<const E*>(gate), gate_ld, kind, P, static_cast<E*>(y), y_ld, static_cast<E*>(h), h_ld, \
                  rstd_post, rstd_pre)
  if (dtype == DET_BF16) {
    DET_NORM_FWD(uint16_t)
  } else {
    DET_NORM_FWD(float)
  }
#undef DET_NORM_FWD
  return check_launch("det_block_norm");
}

extern "C" int det_block_norm_bwd_workspace_size(int64_t T, int64_t D, size_t* bytes) {
  if (!bytes) return set_error(DET_ERR_INVALID_ARG, "block_norm_bwd: bytes is NULL");
  if (int s = check_sizes("block_norm_bwd", T, D)) return s;
  *bytes = ws_bytes_for(T, D);
  return ok();
}

extern "C" int det_block_norm_bwd(const void* dy, int64_t dy_ld, const void* dh, int64_t dh_ld, const void* x,
                                  int64_t x_ld, const void* f, int64_t f_ld, const void* gate, int64_t gate_ld,
                                  int64_t gate_cols, const float* w_post, const float* alpha, const float* w_pre,
                                  const float* rstd_post, const float* rstd_pre, int dtype, int64_t T, int64_t D,
                                  void* dx, int64_t dx_ld, void* df, int64_t df_ld, void* dgate, int64_t dgate_ld,
                                  float* dw_post, float* dalpha, float* dw_pre, void* ws, size_t ws_bytes,
                                  void* stream) {
  const char* what = "block_norm_bwd";
  if (int s = check_sizes(what, T, D)) return s;
  if (int s = check_float_dtype(what, dtype)) return s;
  if (T == 0 || D == 0) return ok();
  if (!dy || !f || !dx || !df) return set_error(DET_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if (gate && gate_cols != 1 && gate_cols != D)
    return set_error(DET_ERR_INVALID_ARG, "%s: gate_cols must be 1 or D, got %lld", what, (long long)gate_cols);
  const bool post = w_post != nullptr, pre = w_pre != nullptr;
  if (pre != (dh != nullptr) || pre != (rstd_pre != nullptr) || pre != (dw_pre != nullptr) || (pre && !x))
    return set_error(DET_ERR_INVALID_ARG, "%s: w_pre, dh, rstd_pre and dw_pre go together (and need x)", what);
  if (post != (rstd_post != nullptr) || post != (dw_post != nullptr))
    return set_error(DET_ERR_INVALID_ARG, "%s: w_post, rstd_post and dw_post go together", what);
  if ((alpha != nullptr) != (dalpha != nullptr))
    return set_error(DET_ERR_INVALID_ARG, "%s: alpha and dalpha go together", what);
  if ((gate != nullptr) != (dgate != nullptr))
    return set_error(DET_ERR_INVALID_ARG, "%s: gate and dgate go together", what);
  const struct {
    const char* name;
    const void* p;
    int64_t ld, cols;
  } rows[] = {{"dy", dy, dy_ld, D}, {"dh", dh, dh_ld, D}, {"x", x, x_ld, D}, {"f", f, f_ld, D},
              {"gate", gate, gate_ld, gate_cols}, {"dx", dx, dx_ld, D}, {"df", df, df_ld, D},
              {"dgate", dgate, dgate_ld, gate_cols}};
  Buf rr[8];
  for (int i = 0; i < 8; ++i) {
    if (int s = check_ld(what, rows[i].name, rows[i].p, rows[i].ld, rows[i].cols, T)) return s;
    rr[i] = buf_rows(rows[i].name, rows[i].p, T, rows[i].cols, rows[i].ld, dtype_size(dtype));
  }
  const size_t need = post || pre || alpha ? ws_bytes_for(T, D) : 0;
  if (int s = check_workspace(ws, ws_bytes, need)) return s;
  const Buf outs[] = {rr[5], rr[6], rr[7],
                      {"dw_post", range1d(dw_post, D * 4)},
                      {"dalpha", range1d(dalpha, D * 4)},
                      {"dw_pre", range1d(dw_pre, D * 4)},
                      {"the workspace", range1d(need ? ws : nullptr, ws_bytes)}};
  const Buf ins[] = {rr[0], rr[1], rr[2], rr[3], rr[4],
                     {"w_post", range1d(w_post, D * 4)},
                     {"alpha", range1d(alpha, D * 4)},
                     {"w_pre", range1d(w_pre, D * 4)},
                     {"rstd_post", range1d(rstd_post, T * 4)},
                     {"rstd_pre", range1d(rstd_pre, T * 4)}};
  if (int s = check_buffers(what, outs, 7, ins, 10)) return s;
  const NormParams P{w_post, alpha, w_pre, 0.0f, static_cast<float>(1.0 / D), T, D};
  const int kind = !gate ? kGateNone : (gate_cols == D ? kGateFull : kGateRow);
  const bool full = kind == kGateFull;
  const int64_t groups = groups_for(T, D, true);
  const dim3 grid(static_cast<uint32_t>(groups));
  const bool past = past_caches(T * D * static_cast<int64_t>(dtype_size(dtype)) * (full ? 3 : 2));
  const hipStream_t st = as_stream(stream);
  auto* slots = need ? reinterpret_cast<float*>(static_cast<char*>(ws) + DET_WS_HEADER_BYTES) : nullptr;
#define DET_NORM_BWD(E)                                                                                              \
  {                                                                                                                  \
    const BwdIn<E> I{static_cast<const E*>(dy), static_cast<const E*>(dh), static_cast<const E*>(x),                 \
                     static_cast<const E*>(f),  static_cast<const E*>(gate), dy_ld, dh_ld, x_ld, f_ld, gate_ld,      \
                     rstd_post, rstd_pre, kind == kGateRow};                                                         \
    DET_NORM_LAUNCH(DET_NORM_BWD_KERNEL, E, I, P, static_cast<E*>(dx), dx_ld, static_cast<E*>(df), df_ld,            \
                    static_cast<E*>(dgate), dgate_ld, slots)                                                         \
  }
  if (dtype == DET_BF16) {
    DET_NORM_BWD(uint16_t)
  } else {
    DET_NORM_BWD(float)
  }
#undef DET_NORM_BWD
  if (need)
    hipLaunchKernelGGL(norm_fold_kernel, dim3(static_cast<uint32_t>(ceil_div(D, 64)), 2), dim3(64 * kFoldWaves), 0, st, slots,
                       static_cast<int>(groups), P, NormGrads{dw_post, dalpha, dw_pre});
  return check_launch("det_block_norm_bwd");
}
