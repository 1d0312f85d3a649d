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
//   dx = D;  dw_pre += sum dh yh;  dalpha += sum D s n
//   dn = D alpha s:  dgate = dn n (1 - s)  (its row sum for a gate per token)
//   fh = f rstd_f:   dw_post += sum dn fh;  df = rstd_f (w_post dn - fh mean(w_post dn fh))   (w_post NULL: df = dn)
//
// A workgroup owns whole rows, eight (or sixteen) consecutive channels per
// thread, so a row's sums are a wave tree and one exchange through LDS, and the
// parameters and the parameter gradients' running sums of a thread's channels
// stay in registers while it walks its rows. The parameter gradients are column
// sums: workgroup b adds rows b, b + G, b + 2G, ... in order into its own slot
// (no atomics), a fold adds the slots in a fixed order and once into the output.
//
// Both directions are bound by the [T, D] tensors: five read or written forward,
// eight backward.
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

__device__ __forceinline__ float sigmoid_f(float g) { return 1.0f / (1.0f + exp_e(-g)); }

enum GateKind { kGateNone = 0, kGateRow = 1, kGateFull = 2 };

struct NormParams {
  const float *w_post, *alpha, *w_pre;  // [D] float32, NULL: not applied
  float eps, inv_d;
  int64_t rows, D;
};

template <int N>
__device__ __forceinline__ void load_param(const float* p, int64_t col, int64_t n, float (&v)[N]) {
  if (p) {
    load8(p + col, n, 0.0f, v);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = 1.0f;
  }
}

template <typename T, int THREADS, int NV>
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
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (i * THREADS + threadIdx.x) * 8;
    float al[8];
    load_param(P.w_post, col, P.D - col, wp[i]);
    load_param(P.alpha, col, P.D - col, al);
    load_param(P.w_pre, col, P.D - col, wq[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) wp[i][j] *= al[j];
  }
  for (int64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
    float xv[NV][8], fv[NV][8], gv[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (i * THREADS + threadIdx.x) * 8;
      load8(f + r * ld_f + col, P.D - col, 0.0f, fv[i]);
      load8(x + r * ld_x + col, P.D - col, 0.0f, xv[i]);
      if (gate_kind == kGateFull) load8(gate + r * ld_g + col, P.D - col, 0.0f, gv[i]);
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
      const int64_t col = (i * THREADS + threadIdx.x) * 8;
      store8(y + r * ld_y + col, P.D - col, xv[i]);
    }
    if (pre) {
      const float rq = 1.0f / sqrtf(block_sum<THREADS>(q, buf[1]) * P.inv_d + P.eps);
      if (threadIdx.x == 0) rstd_pre[r] = rq;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t col = (i * THREADS + threadIdx.x) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) xv[i][j] = xv[i][j] * rq * wq[i][j];
        store8(h + r * ld_h + col, P.D - col, xv[i]);
      }
    }
    // with one sum per row the same buffer serves every row
    if (THREADS > 64 && post != pre) __syncthreads();
  }
}

// Rows a workgroup's slot holds: dw_post, dalpha, dw_pre, in this order.
template <typename T, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void norm_bwd_kernel(const T* __restrict__ dy, int64_t ld_dy,
                                                           const T* __restrict__ dh, int64_t ld_dh,
                                                           const T* __restrict__ x, int64_t ld_x,
                                                           const T* __restrict__ f, int64_t ld_f,
                                                           const T* __restrict__ gate, int64_t ld_g, int gate_kind,
                                                           NormParams P, const float* __restrict__ rstd_post,
                                                           const float* __restrict__ rstd_pre, T* __restrict__ dx,
                                                           int64_t ld_dx, T* __restrict__ df, int64_t ld_df,
                                                           T* __restrict__ dgate, int64_t ld_dg,
                                                           float* __restrict__ slots) {
  __shared__ float buf[2][THREADS / 64];
  const bool post = P.w_post != nullptr, pre = P.w_pre != nullptr;
  const bool second = post || gate_kind == kGateRow;  // a second sum over the row is needed
  float wp[NV][8], al[NV][8], wq[NV][8];
  float g_post[NV][8] = {}, g_alpha[NV][8] = {}, g_pre[NV][8] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (i * THREADS + threadIdx.x) * 8;
    load_param(P.w_post, col, P.D - col, wp[i]);
    load_param(P.alpha, col, P.D - col, al[i]);
    load_param(P.w_pre, col, P.D - col, wq[i]);
  }
  for (int64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
    float d[NV][8], fh[NV][8], s[NV][8], yh[NV][8], u[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (i * THREADS + threadIdx.x) * 8, n = P.D - col;
      load8(f + r * ld_f + col, n, 0.0f, fh[i]);
      load8(dy + r * ld_dy + col, n, 0.0f, d[i]);
      if (gate_kind == kGateFull) load8(gate + r * ld_g + col, n, 0.0f, s[i]);
      if (pre) {
        load8(x + r * ld_x + col, n, 0.0f, yh[i]);
        load8(dh + r * ld_dh + col, n, 0.0f, u[i]);
      }
    }
    const float s_row = gate_kind == kGateRow ? sigmoid_f(to_f32(gate[r * ld_g])) : 1.0f;
    const float rp = post ? rstd_post[r] : 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        fh[i][j] *= rp;
        s[i][j] = gate_kind == kGateFull ? sigmoid_f(s[i][j]) : s_row;
      }
    if (pre) {
      const float rq = rstd_pre[r];
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          yh[i][j] = (yh[i][j] + fh[i][j] * (wp[i][j] * al[i][j]) * s[i][j]) * rq;
          g_pre[i][j] += u[i][j] * yh[i][j];
          u[i][j] *= wq[i][j];
          q += u[i][j] * yh[i][j];
        }
      const float mean = block_sum<THREADS>(q, buf[0]) * P.inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) d[i][j] += rq * (u[i][j] - yh[i][j] * mean);
    }
    // d = the gradient of y; from here u = dn = d alpha s
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (i * THREADS + threadIdx.x) * 8;
      store8(dx + r * ld_dx + col, P.D - col, d[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float ds = d[i][j] * s[i][j];
        g_alpha[i][j] += ds * (fh[i][j] * wp[i][j]);
        const float dn = ds * al[i][j];
        g_post[i][j] += dn * fh[i][j];
        u[i][j] = dn * wp[i][j];
        q += u[i][j] * fh[i][j];
      }
      if (gate_kind == kGateFull) {
        float dg[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) dg[j] = u[i][j] * fh[i][j] * (1.0f - s[i][j]);
        store8(dgate + r * ld_dg + col, P.D - col, dg);
      }
    }
    if (second) {
      const float tot = block_sum<THREADS>(q, buf[1]);
      if (gate_kind == kGateRow && threadIdx.x == 0) dgate[r * ld_dg] = from_f32<T>(tot * (1.0f - s_row));
      if (post) {
        const float mean = tot * P.inv_d;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) u[i][j] = rp * (u[i][j] - fh[i][j] * mean);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = (i * THREADS + threadIdx.x) * 8;
      store8(df + r * ld_df + col, P.D - col, u[i]);
    }
    if (THREADS > 64 && second != pre) __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = (i * THREADS + threadIdx.x) * 8, n = P.D - col;
    float* o = slots + static_cast<int64_t>(blockIdx.x) * 3 * P.D + col;
    if (post) store8(o, n, g_post[i]);
    if (P.alpha) store8(o + P.D, n, g_alpha[i]);
    if (pre) store8(o + 2 * P.D, n, g_pre[i]);
  }
}

// Workgroup (64 columns, parameter): wave w adds slots w, w + 4, ... in order,
// the four sums meet left to right, one add into the output.
struct NormGrads {
  float* g[3];
};
__global__ __launch_bounds__(256) void norm_fold_kernel(const float* __restrict__ slots, int n_slots, int64_t D,
                                                        NormGrads G) {
  __shared__ float part[4][64];
  float* out = G.g[blockIdx.y];
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const float* p = slots + blockIdx.y * D + col;
  float t = 0.0f;
  if (col < D)
    for (int b = wave; b < n_slots; b += 64) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = b + 4 * i < n_slots ? p[static_cast<int64_t>(b + 4 * i) * 3 * D] : 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) t += v[i];
    }
  part[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && col < D) out[col] += ((part[0][lane] + part[1][lane]) + part[2][lane]) + part[3][lane];
}

int threads_for(int64_t D) {
  int t = 64;
  while (t < 1024 && t * 8 < D) t *= 2;
  return t;
}

// Workgroups of a launch: every compute unit's 2048 threads, twice over for the
// forward (no per-workgroup cost beyond the parameters), once for the backward,
// whose every workgroup writes a slot of 12 bytes per channel.
int64_t groups_for(int64_t T, int64_t D, bool bwd) {
  const int64_t g = 256 * (2048 / threads_for(D)) * (bwd ? 1 : 2) / (bwd && D > 512 ? 2 : 1);
  return T < g ? T : g;
}
size_t ws_bytes_for(int64_t T, int64_t D) {
  return T == 0 || D == 0 ? 0
                          : DET_WS_HEADER_BYTES + align_up(static_cast<size_t>(groups_for(T, D, true) * 3 * D) * 4, 256);
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

#define DET_NORM_LAUNCH(KERNEL, T, ...)                                                                            \
  switch (D > 8192 ? 2048 : threads_for(D)) {                                                                      \
    case 64: hipLaunchKernelGGL((KERNEL<T, 64, 1>), grid, dim3(64), 0, st, __VA_ARGS__); break;                    \
    case 128: hipLaunchKernelGGL((KERNEL<T, 128, 1>), grid, dim3(128), 0, st, __VA_ARGS__); break;                 \
    case 256: hipLaunchKernelGGL((KERNEL<T, 256, 1>), grid, dim3(256), 0, st, __VA_ARGS__); break;                 \
    case 512: hipLaunchKernelGGL((KERNEL<T, 512, 1>), grid, dim3(512), 0, st, __VA_ARGS__); break;                 \
    case 1024: hipLaunchKernelGGL((KERNEL<T, 1024, 1>), grid, dim3(1024), 0, st, __VA_ARGS__); break;              \
    default: hipLaunchKernelGGL((KERNEL<T, 1024, 2>), grid, dim3(1024), 0, st, __VA_ARGS__); break;                \
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
  Range rr[5];
  for (int i = 0; i < 5; ++i) {
    if (int s = check_ld(what, rows[i].name, rows[i].p, rows[i].ld, rows[i].cols, T)) return s;
    rr[i] = range2d(rows[i].p, T, rows[i].cols, rows[i].ld, dtype_size(dtype));
  }
  const Buf outs[] = {{"y", rr[3]}, {"h", rr[4]}, {"rstd_post", range1d(rstd_post, T * 4)},
                      {"rstd_pre", range1d(rstd_pre, T * 4)}};
  const Buf ins[] = {{"x", rr[0]}, {"f", rr[1]}, {"gate", rr[2]}, {"w_post", range1d(w_post, D * 4)},
                     {"alpha", range1d(alpha, D * 4)}, {"w_pre", range1d(w_pre, D * 4)}};
  if (int s = check_overlaps(what, outs, 4, ins, 6)) return s;
  const NormParams P{w_post, alpha, w_pre, static_cast<float>(eps), static_cast<float>(1.0 / D), T, D};
  const int kind = !gate ? kGateNone : (gate_cols == D ? kGateFull : kGateRow);
  const dim3 grid(static_cast<uint32_t>(groups_for(T, D, false)));
  const hipStream_t st = as_stream(stream);
#define DET_NORM_FWD(E)                                                                                             \
  DET_NORM_LAUNCH(norm_fwd_kernel, E, static_cast<const E*>(x), x_ld, static_cast<const E*>(f), f_ld,               \
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
  Range rr[8];
  for (int i = 0; i < 8; ++i) {
    if (int s = check_ld(what, rows[i].name, rows[i].p, rows[i].ld, rows[i].cols, T)) return s;
    rr[i] = range2d(rows[i].p, T, rows[i].cols, rows[i].ld, dtype_size(dtype));
  }
  const size_t need = post || pre || alpha ? ws_bytes_for(T, D) : 0;
  if (int s = check_workspace(ws, ws_bytes, need)) return s;
  const Buf outs[] = {{"dx", rr[5]},
                      {"df", rr[6]},
                      {"dgate", rr[7]},
                      {"dw_post", range1d(dw_post, D * 4)},
                      {"dalpha", range1d(dalpha, D * 4)},
                      {"dw_pre", range1d(dw_pre, D * 4)},
                      {"the workspace", range1d(need ? ws : nullptr, ws_bytes)}};
  const Buf ins[] = {{"dy", rr[0]}, {"dh", rr[1]}, {"x", rr[2]}, {"f", rr[3]}, {"gate", rr[4]},
                     {"w_post", range1d(w_post, D * 4)}, {"alpha", range1d(alpha, D * 4)},
                     {"w_pre", range1d(w_pre, D * 4)}, {"rstd_post", range1d(rstd_post, T * 4)},
                     {"rstd_pre", range1d(rstd_pre, T * 4)}};
  if (int s = check_overlaps(what, outs, 7, ins, 10)) return s;
  const NormParams P{w_post, alpha, w_pre, 0.0f, static_cast<float>(1.0 / D), T, D};
  const int kind = !gate ? kGateNone : (gate_cols == D ? kGateFull : kGateRow);
  const int64_t groups = groups_for(T, D, true);
  const dim3 grid(static_cast<uint32_t>(groups));
  const hipStream_t st = as_stream(stream);
  auto* slots = need ? reinterpret_cast<float*>(static_cast<char*>(ws) + DET_WS_HEADER_BYTES) : nullptr;
#define DET_NORM_BWD(E)                                                                                               \
  DET_NORM_LAUNCH(norm_bwd_kernel, E, static_cast<const E*>(dy), dy_ld, static_cast<const E*>(dh), dh_ld,             \
                  static_cast<const E*>(x), x_ld, static_cast<const E*>(f), f_ld, static_cast<const E*>(gate), gate_ld, \
                  kind, P, rstd_post, rstd_pre, static_cast<E*>(dx), dx_ld, static_cast<E*>(df), df_ld,               \
                  static_cast<E*>(dgate), dgate_ld, slots)
  if (dtype == DET_BF16) {
    DET_NORM_BWD(uint16_t)
  } else {
    DET_NORM_BWD(float)
  }
#undef DET_NORM_BWD
  if (need)
    hipLaunchKernelGGL(norm_fold_kernel, dim3(static_cast<uint32_t>(ceil_div(D, 64)), 3), dim3(256), 0, st, slots,
                       static_cast<int>(groups), D, NormGrads{{dw_post, dalpha, dw_pre}});
  return check_launch("det_block_norm_bwd");
}
