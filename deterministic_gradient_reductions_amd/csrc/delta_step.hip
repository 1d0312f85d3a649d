// det_delta_rule_step: one token per row of a batch through the gated delta rule,
// against a cache of float32 states that is updated in place.
//
//   S' = exp(g) S;  u = beta (v - S'^T k);  S <- S' + k u^T;  o = scale S^T q = scale (S'^T q + (k . q) u)
//
// so the two products with S' run over the state as it was read, once, and the state is
// written once: 8 bytes of memory per element are all there is to do. A thread holds
// four columns of some rows; sums over rows meet in LDS in one fixed order.
//
// Rows that name one slot are tokens of one sequence in row order: the first of them
// owns the slot and takes the others' tokens after its own, with the state in registers.
#include "delta.hpp"

namespace detgrad {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct StepArgs {
  Heads<const T> q, k, v;
  Heads<T> o;
  const float* g;
  const T* beta;
  float* state;
  const int32_t* slots;
  int64_t g_ld, beta_ld, N;
  int B, Hk, H, dk, dv;
  float scale;
};

// Workgroup (h, b, block): columns VB block .. of head h of row b. Lanes cover VB / 4
// groups of four columns; the others, rows row0, row0 + kGroups, ... of the state.
template <typename T, int VB>
__global__ __launch_bounds__(kThreads) void delta_step_kernel(StepArgs<T> A) {
  constexpr int kCols = VB / 4, kGroups = kThreads / kCols, kRows = kDeltaMaxDim / kGroups;
  __shared__ float lk[kDeltaMaxDim], lq[kDeltaMaxDim];
  __shared__ f32x4 part[2][kGroups][kCols];
  __shared__ float dots[kThreads / 64];
  __shared__ int next_row;
  const int h = blockIdx.x, b = blockIdx.y, hk = h / (A.H / A.Hk);
  const int cg = threadIdx.x % kCols, rg = threadIdx.x / kCols, col = blockIdx.z * VB + 4 * cg;
  const int nv = A.dv - col;  // columns of this thread, up to four
  const int64_t slot = A.slots ? A.slots[b] : b;
  if (slot < 0 || slot >= A.N) {
    if (rg == 0 && nv > 0) store4(A.o.row(b, h) + col, nv, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
    return;
  }
  float* p = A.state + (slot * A.H + h) * (static_cast<int64_t>(A.dk) * A.dv);
  const bool whole = A.dv % 4 == 0;
  f32x4 s[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int d = i * kGroups + rg;
    s[i] = load4(p + static_cast<int64_t>(d < A.dk ? d : 0) * A.dv, col, A.dv, whole);
  }
  if (A.slots) {  // an earlier row of this slot: that row's workgroup takes this token
    int before = 0;
    for (int j = threadIdx.x; j < b; j += kThreads) before |= A.slots[j] == slot;
    if (__syncthreads_or(before)) return;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) s[i] = i * kGroups + rg < A.dk ? s[i] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int row = b;;) {
    float x = 0.0f, y = 0.0f;
    if (threadIdx.x < kDeltaMaxDim) {
      if (static_cast<int>(threadIdx.x) < A.dk) {
        x = to_f32(A.k.row(row, hk)[threadIdx.x]);
        y = to_f32(A.q.row(row, hk)[threadIdx.x]);
      }
      lk[threadIdx.x] = x;
      lq[threadIdx.x] = y;
    }
    const f32x4 v = load4(A.v.row(row, h), col, A.dv, whole);
    const float gt = A.g[row * A.g_ld + h], bt = to_f32(A.beta[row * A.beta_ld + h]);
    const float dot = lanes_sum<64>(x * y);
    if ((threadIdx.x & 63) == 0) dots[threadIdx.x >> 6] = dot;
    if (threadIdx.x == 0) next_row = A.B;
    __syncthreads();
    const float a = exp_e(gt);
    f32x4 pk{}, pq{};
    float kd[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int d = i * kGroups + rg;
      kd[i] = lk[d];
      const float qd = lq[d];
      s[i] *= a;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        pk[j] = __builtin_fmaf(kd[i], s[i][j], pk[j]);
        pq[j] = __builtin_fmaf(qd, s[i][j], pq[j]);
      }
    }
    part[0][rg][cg] = pk;
    part[1][rg][cg] = pq;
    if (A.slots) {
      int next = A.B;
      for (int j = row + 1 + threadIdx.x; j < A.B; j += kThreads)
        if (A.slots[j] == slot) {
          next = j;
          break;
        }
      if (next < A.B) atomicMin(&next_row, next);  // a minimum: the order does not matter
    }
    __syncthreads();
    pk = part[0][0][cg];
    pq = part[1][0][cg];
#pragma unroll 8
    for (int i = 1; i < kGroups; ++i) {
      pk += part[0][i][cg];
      pq += part[1][i][cg];
    }
    f32x4 u, o;
    const float kq = dots[0] + dots[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = bt * (v[j] - pk[j]);
      o[j] = A.scale * __builtin_fmaf(kq, u[j], pq[j]);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = __builtin_fmaf(kd[i], u[j], s[i][j]);
    if (rg == 0 && nv > 0) store4(A.o.row(row, h) + col, nv, o);
    const int to = next_row;
    if (!A.slots || to >= A.B) break;
    __syncthreads();  // everyone has read the sums and the next row
    row = to;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int d = i * kGroups + rg;
    if (d < A.dk && nv > 0) store4(p + static_cast<int64_t>(d) * A.dv + col, nv, s[i]);
  }
}

template <typename T>
void launch_step(const StepArgs<T>& A, hipStream_t st) {
  // the widest workgroup that leaves two for each compute unit
  const int64_t rows = static_cast<int64_t>(A.B) * A.H;
  const int vb = rows >= 512 && A.dv > 64 ? 128 : (rows * ceil_div(A.dv, 64) >= 512 && A.dv > 32 ? 64 : 32);
  const dim3 grid(static_cast<uint32_t>(A.H), static_cast<uint32_t>(A.B), static_cast<uint32_t>(ceil_div(A.dv, vb)));
  if (vb == 128) hipLaunchKernelGGL((delta_step_kernel<T, 128>), grid, dim3(kThreads), 0, st, A);
  else if (vb == 64) hipLaunchKernelGGL((delta_step_kernel<T, 64>), grid, dim3(kThreads), 0, st, A);
  else hipLaunchKernelGGL((delta_step_kernel<T, 32>), grid, dim3(kThreads), 0, st, A);
}

}  // namespace
}  // namespace detgrad

using namespace detgrad;

extern "C" int det_delta_rule_step(const void* q, int64_t q_st, int64_t q_sh, const void* k, int64_t k_st, int64_t k_sh,
                                   const void* v, int64_t v_st, int64_t v_sh, const float* g, int64_t g_ld,
                                   const void* beta, int64_t beta_ld, int dtype, int64_t B, int64_t Hk, int64_t H,
                                   int64_t dk, int64_t dv, double scale, float* state, int64_t N, const int32_t* slots,
                                   void* o, int64_t o_st, int64_t o_sh, void* stream) {
  const char* what = "delta_rule_step";
  if (int s = delta_check_sizes(what, dtype, B, 0, Hk, H, dk, dv)) return s;
  if (!(scale > -1e30 && scale < 1e30)) return set_error(DET_ERR_INVALID_ARG, "%s: scale must be finite", what);
  if (N < 0 || N > 0x7FFFFFFF) return set_error(DET_ERR_INVALID_ARG, "%s: N must lie in [0, 2^31)", what);
  if (B > 65535) return set_error(DET_ERR_UNSUPPORTED, "%s: B must be <= 65535", what);
  if (!slots && B > N) return set_error(DET_ERR_INVALID_ARG, "%s: without slots the cache needs a state per row", what);
  if (H * B * 4 * kThreads > 0xFFFFFFFF) return set_error(DET_ERR_UNSUPPORTED, "%s: problem too large", what);
  if (B == 0) return ok();
  if (!q || !k || !v || !g || !beta || !o || (N > 0 && !state))
    return set_error(DET_ERR_INVALID_ARG, "%s: NULL pointer", what);
  const size_t es = dtype_size(dtype);
  Buf bq, bk, bv, bo;
  if (int s = delta_buf(what, "q", q, B, Hk, dk, q_st, q_sh, es, bq)) return s;
  if (int s = delta_buf(what, "k", k, B, Hk, dk, k_st, k_sh, es, bk)) return s;
  if (int s = delta_buf(what, "v", v, B, H, dv, v_st, v_sh, es, bv)) return s;
  if (int s = delta_buf(what, "o", o, B, H, dv, o_st, o_sh, es, bo)) return s;
  if (B > 1 && (g_ld < H || beta_ld < H)) return set_error(DET_ERR_INVALID_ARG, "%s: row stride of g or beta < H", what);
  if (g_ld > (int64_t(1) << 44) / B || beta_ld > (int64_t(1) << 44) / B)
    return set_error(DET_ERR_UNSUPPORTED, "%s: g or beta is too large", what);
  const Buf outs[] = {bo, {"state", range1d(state, static_cast<size_t>(N) * H * dk * dv * 4)}};
  const Buf ins[] = {bq, bk, bv, buf_rows("g", g, B, H, B > 1 ? g_ld : H, 4),
                     buf_rows("beta", beta, B, H, B > 1 ? beta_ld : H, es), {"slots", range1d(slots, B * 4)}};
  if (int s = check_buffers(what, outs, 2, ins, 6)) return s;
#define DET_DELTA_STEP(E)                                                                                            \
  launch_step<E>(StepArgs<E>{{static_cast<const E*>(q), q_st, q_sh}, {static_cast<const E*>(k), k_st, k_sh},         \
                             {static_cast<const E*>(v), v_st, v_sh}, {static_cast<E*>(o), o_st, o_sh}, g,            \
                             static_cast<const E*>(beta), state, slots, g_ld, beta_ld, N, (int)B, (int)Hk, (int)H,   \
                             (int)dk, (int)dv, static_cast<float>(scale)},                                           \
                 as_stream(stream))
  if (dtype == DET_BF16) DET_DELTA_STEP(uint16_t);
  else DET_DELTA_STEP(float);
#undef DET_DELTA_STEP
  return check_launch("det_delta_rule_step");
}
