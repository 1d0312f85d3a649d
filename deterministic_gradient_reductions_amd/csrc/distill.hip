// det_topk_distill / det_topk_distill_bwd: distillation from a teacher's top
// logits, per token t over a vocabulary of V words.
//
//   x = z / tau,  lse = log sum_v exp(x_v)
//   q = softmax of teacher / tau over the valid slots (0 <= id < V)
//   loss = sum_k q_k (log q_k - x[id_k] + lse)          (slots with q_k = 0 add nothing)
//   dz_v = dloss / tau (exp(x_v - lse) - sum of q_k over the slots with id_k = v)
//
// A row without teacher mass (no valid slot, or only -inf there) has loss 0 and
// a zero gradient row, and so has a row whose dloss is 0, whatever its logits.
//
// Forward: one pass over the row with a running maximum and sum per lane
// (rescaled when the maximum grows), joined over the lanes, the waves and, for
// few very long rows, the workgroups that share a row, always in one fixed
// order. Backward: dz of a piece of the row is written in one streaming pass,
// then the workgroup rewrites the at most K elements that a teacher slot names.
// The slots' words and logits are fetched into LDS while the row streams.
// Both are bound by the logits' bytes (8192 x 131072 bf16: forward 359 us, 6.0 TB/s;
// backward 726 us, 5.9 TB/s); the backward takes the rows in reverse order, so
// that after a forward it first meets the rows still cached (18 us there).
#include "rowops.hpp"

namespace detgrad {
namespace {

constexpr int kMaxK = 1024;
// 16-byte loads of a lane in flight together: in the forward's main loop, in the
// loop that takes most of what is left, in the backward's.
constexpr int kUnroll = 8, kUnrollRest = 2, kBwdUnroll = 4;
constexpr int kBwdThreads = 256;
// A float32 lse below 2^10 in size is off by at most 2^-15, and so is p taken from
// it. A larger one (every word masked by -1e4, or by the type's lowest value, where
// nothing of log s is left in it) is not used: the backward forms such a row's
// maximum and sum again, which costs each of its pieces two reads of the row.
constexpr float kFarLse = 0x1p10f;

// Everything below is in units of log2: x2 = x log2(e) = c z with
// c = log2(e) / tau, formed by one fused step against the reference, so only
// the difference is rounded. MaxSum: the reference m (a rounded maximum of c z,
// at least kLow) and s = sum of 2^(c z - m). m is off from the true maximum by up
// to 2^-25 |m|, which cancels as long as it is small: where |m| reaches 2^20 it
// could take s past float32. So a lane that has met nothing but masked words (-inf,
// the type's lowest value, -1e30) stays at kLow, against which they count 0, and a
// row whose own reference is out of (kLow, -kLow) is summed another way (far_row).
constexpr float kLow = -0x1p20f;
struct MaxSum {
  float m, s;
};

template <int N>
struct Int {
  static constexpr int value = N;
};

__device__ __forceinline__ float pow2(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ bool is_far(MaxSum a) { return !(a.m > kLow && a.m < -kLow); }

__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b) {
  const float m = fmaxf(a.m, b.m);
  return {m, a.s * pow2(a.m - m) + b.s * pow2(b.m - m)};
}

// Over groups of W lanes.
template <int W>
__device__ __forceinline__ MaxSum lanes_join(MaxSum a) {
#pragma unroll
  for (int d = 1; d < W; d <<= 1) {
    const MaxSum o{__shfl_xor(a.m, d), __shfl_xor(a.s, d)};
    a = join(a, o);
  }
  return a;
}

// Adds 8 N elements: their own sum first (a short tree of chains), then the
// running sum, so the running chain is one add per 8 N elements long.
template <int N>
__device__ __forceinline__ void push(MaxSum& a, const float (&v)[N][8], float c) {
  float m = -__builtin_inff();
#pragma unroll
  for (int u = 0; u < N; ++u)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, v[u][j]);
  m = fmaxf(a.m, m * c);
  float s[4] = {};
#pragma unroll
  for (int u = 0; u < N; ++u)
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j & 3] += pow2(__builtin_fmaf(v[u][j], c, -m));
  a = {m, a.s * pow2(a.m - m) + ((s[0] + s[1]) + (s[2] + s[3]))};
}

// What turns a logit of the row into x - lse: (c (z - z0) - m) ln 2 - log s, whose
// first part is one fused step, so log s is not lost where |lse| is large. z0 = 0
// but for far rows. (A masked word's c z may leave float32 where its z / tau does
// not: that is then the whole of the difference.)
struct Norm {
  float z0, m, logs;
  __device__ __forceinline__ float log_p(float z, float it) const {
    const float d = __builtin_fmaf(z - z0, it * kLog2e, -m);
    return (d == -__builtin_inff() ? (z - z0) * it - m * kLn2 : d * kLn2) - logs;
  }
};

// The same for a row whose reference is far from 0 (every logit masked by a large
// negative number, or one large positive one), by the whole workgroup in two
// passes over the row: the maximum of z itself, then the sum against it. Rows of
// nothing but -inf and rows with +inf come here too and keep the values that the
// formulas give them. `part` has one float per wave.
template <typename T, int THREADS>
__device__ __forceinline__ Norm far_row(const T* __restrict__ p, int64_t V, float c, float* part) {
  constexpr int kWaves = THREADS / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  keep_branch();
  float m = -__builtin_inff();
  for (int64_t i = threadIdx.x * 8; i < V; i += THREADS * 8) {
    float v[8];
    load8(p + i, V - i, -__builtin_inff(), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, v[j]);
  }
  m = lanes_max<64>(m);
  __syncthreads();
  if (lane == 0) part[wave] = m;
  __syncthreads();
  for (int w = 0; w < kWaves; ++w) m = fmaxf(m, part[w]);
  const float r = m == -__builtin_inff() ? 0.0f : m;
  float s = 0.0f;
  for (int64_t i = threadIdx.x * 8; i < V; i += THREADS * 8) {
    float v[8];
    load8(p + i, V - i, -__builtin_inff(), v);
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) t += pow2((v[j] - r) * c);
    s += t;
  }
  s = lanes_sum<64>(s);
  __syncthreads();
  if (lane == 0) part[wave] = s;
  __syncthreads();
  s = part[0];
  for (int w = 1; w < kWaves; ++w) s += part[w];
  return {m, 0.0f, logf(s)};
}

// A row's teacher slots in LDS: the word, the teacher's logit (-inf for an invalid
// slot, which has no weight either way) and the student's.
struct Slots {
  int32_t id[kMaxK];
  float t[kMaxK], x[kMaxK];
};
// Slots k of the row with lo <= id < hi get their student logit (others 0); a
// slot outside [0, V) gets the word -1.
template <typename T, typename TT, int THREADS>
__device__ __forceinline__ void fetch_slots(Slots& S, const int32_t* __restrict__ ids, const TT* __restrict__ t, int K,
                                            int64_t V, const T* __restrict__ z, int64_t lo, int64_t hi) {
  for (int k = threadIdx.x; k < K; k += THREADS) {
    const int32_t id = ids[k];
    const float tk = to_f32(t[k]);
    const bool valid = id >= 0 && id < V, in = id >= lo && id < hi;
    const float x = to_f32(z[in ? id : lo]);
    S.id[k] = valid ? id : -1;
    S.t[k] = valid ? tk : -__builtin_inff();
    S.x[k] = in ? x : 0.0f;
  }
}

// The teacher's softmax over the valid slots, by one wave: t is at most m (0 if
// no slot is above -inf), sum = sum exp((t - m) / tau); 0 for a row without mass.
struct Teacher {
  float m, sum;
};
__device__ __forceinline__ Teacher teacher_row(const Slots& S, int K, float it) {
  const int lane = threadIdx.x & 63;
  float m = -__builtin_inff();
  for (int k = lane; k < K; k += 64) m = fmaxf(m, S.t[k]);
  m = lanes_max<64>(m);
  m = m == -__builtin_inff() ? 0.0f : m;
  float s = 0.0f;
  for (int k = lane; k < K; k += 64) s += exp_e((S.t[k] - m) * it);
  return {m, lanes_sum<64>(s)};
}

// Moves the slots whose words lie in [lo, hi) to the front, in slot order, with
// their q in place of t; by one wave, with no other reading S.t or S.x. Returns
// their number.
__device__ __forceinline__ int gather_slots(Slots& S, int K, Teacher q, float it, int64_t lo, int64_t hi) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int k0 = 0; k0 < K; k0 += 64) {
    const int k = k0 + lane < K ? k0 + lane : K - 1;
    const int32_t id = S.id[k];
    const float t = S.t[k], x = S.x[k];
    const bool in = k0 + lane < K && id >= lo && id < hi;
    const uint64_t mask = __ballot(in);
    const int to = n + __popcll(mask & ((uint64_t(1) << lane) - 1));  // <= k0 + lane: only slots already read
    if (in) {
      S.id[to] = id;
      S.t[to] = exp_e((t - q.m) * it) / q.sum;
      S.x[to] = x;
    }
    n += __popcll(mask);
  }
  return n;
}

// loss and lse of a row, by one wave.
__device__ __forceinline__ void finish_row(const Norm& n, const Slots& S, int K, float it,
                                           float* __restrict__ loss, float* __restrict__ lse) {
  const int lane = threadIdx.x & 63;
  const Teacher q = teacher_row(S, K, it);
  float tot = 0.0f;
  const float inv = 1.0f / q.sum, logsum = logf(q.sum);
  for (int k = lane; k < K; k += 64) {
    const float d = (S.t[k] - q.m) * it, qk = exp_e(d) * inv;
    // (a NaN q_k or an empty row's 0 / 0 does not take the q_k = 0 way out)
    if (q.sum != 0.0f && qk != 0.0f) tot += qk * ((d - logsum) - n.log_p(S.x[k], it));
  }
  tot = lanes_sum<64>(tot);
  if (lane == 0) {
    *loss = tot;
    *lse = __builtin_fmaf(n.z0, it, n.m * kLn2) + n.logs;
  }
}

// Workgroup b: piece b % n_split of row b / n_split, columns [c0, c0 + piece).
template <typename T, typename TT, int THREADS>
__global__ __launch_bounds__(THREADS) void distill_fwd_kernel(const T* __restrict__ z, int64_t ld, int64_t V,
                                                              const int32_t* __restrict__ ids, int64_t ids_ld,
                                                              const TT* __restrict__ teacher, int64_t t_ld, int K,
                                                              float it, int n_split, int64_t piece,
                                                              MaxSum* __restrict__ slots, float* __restrict__ loss,
                                                              float* __restrict__ lse) {
  constexpr int kWaves = THREADS / 64, kStep = THREADS * 8;
  __shared__ MaxSum part[kWaves];
  __shared__ float far_part[kWaves];
  __shared__ Slots S;
  const int64_t row = blockIdx.x / n_split, c0 = (blockIdx.x % n_split) * piece;
  const int64_t c1 = c0 + piece < V ? c0 + piece : V;
  const T* p = z + row * ld;
  const float c = it * kLog2e;
  if (n_split == 1) fetch_slots<T, TT, THREADS>(S, ids + row * ids_ld, teacher + row * t_ld, K, V, p, 0, V);
  MaxSum a{kLow, 0.0f};
  int64_t i = c0;
  const auto stream = [&](auto unroll) {
    constexpr int U = decltype(unroll)::value;
    for (; i + U * kStep <= c1; i += U * kStep) {
      Raw8<T> raw[U];
      float v[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u].load(p + i + u * kStep + threadIdx.x * 8);
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u].get(v[u]);
      push<U>(a, v, c);
    }
  };
  stream(Int<kUnroll>{});
  stream(Int<kUnrollRest>{});
  for (; i < c1; i += kStep) {
    float v[1][8];
    const int64_t k = i + threadIdx.x * 8;
    load8(p + k, c1 - k, -__builtin_inff(), v[0]);
    push<1>(a, v, c);
  }
  a = lanes_join<64>(a);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
  __syncthreads();
  a = lanes_join<kWaves>(part[threadIdx.x % kWaves]);  // every wave's value once in each group of kWaves lanes
  if (n_split > 1) {
    if (threadIdx.x == 0) slots[blockIdx.x] = a;
    return;
  }
  Norm n{0.0f, a.m, logf(a.s)};
  if (is_far(a)) n = far_row<T, THREADS>(p, V, c, far_part);  // (the same in every wave)
  if (threadIdx.x < 64) finish_row(n, S, K, it, loss + row, lse + row);
}

// One workgroup per row joins the row's slots.
template <typename T, typename TT>
__global__ __launch_bounds__(256) void distill_join_kernel(const T* __restrict__ z, int64_t ld, int64_t V,
                                                           const int32_t* __restrict__ ids, int64_t ids_ld,
                                                           const TT* __restrict__ teacher, int64_t t_ld, int K,
                                                           float it, int n_split, const MaxSum* __restrict__ slots,
                                                           float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ Slots S;
  __shared__ float far_part[4];
  const int64_t row = blockIdx.x;
  const T* p = z + row * ld;
  const float c = it * kLog2e;
  fetch_slots<T, TT, 256>(S, ids + row * ids_ld, teacher + row * t_ld, K, V, p, 0, V);
  MaxSum a{kLow, 0.0f};
  for (int i = threadIdx.x & 63; i < n_split; i += 64) a = join(a, slots[row * n_split + i]);
  a = lanes_join<64>(a);
  __syncthreads();
  Norm n{0.0f, a.m, logf(a.s)};
  if (is_far(a)) n = far_row<T, 256>(p, V, c, far_part);
  if (threadIdx.x < 64) finish_row(n, S, K, it, loss + row, lse + row);
}

template <typename T, typename TT, bool PAST>
__global__ __launch_bounds__(kBwdThreads) void distill_bwd_kernel(T* __restrict__ dz, int64_t ld_d,
                                                                  const T* __restrict__ z, int64_t ld, int64_t V,
                                                                  const int32_t* __restrict__ ids, int64_t ids_ld,
                                                                  const TT* __restrict__ teacher, int64_t t_ld, int K,
                                                                  float it, int n_split, int64_t piece,
                                                                  const float* __restrict__ lse,
                                                                  const float* __restrict__ dloss) {
  constexpr int kStep = kBwdThreads * 8;
  __shared__ Slots S;
  __shared__ int n_slots;
  __shared__ float far_part[kBwdThreads / 64];
  const uint32_t b = gridDim.x - 1 - blockIdx.x;
  const int64_t row = b / n_split, at = (b % n_split) * piece;
  const T* p = z + row * ld;
  T* o = dz + row * ld_d;
  // The pieces start on 128-byte lines of dz, so that a wave's stores fill whole lines (rows of an odd V start
  // anywhere); the first takes the `lead` elements before the first line too, one per thread.
  const int64_t first = (-reinterpret_cast<uintptr_t>(o) & 127) / sizeof(T), lead = first < V ? first : V;
  const int64_t c0 = at ? lead + at : 0, c1 = lead + at + piece < V ? lead + at + piece : V;
  if (c0 >= c1) return;
  fetch_slots<T, TT, kBwdThreads>(S, ids + row * ids_ld, teacher + row * t_ld, K, V, p, c0, c1);
  const float a = dloss[row] * it, l = lse[row];
  __syncthreads();
  const Teacher q = teacher_row(S, K, it);  // the same in every wave
  if (a == 0.0f || q.sum == 0.0f) {
    const float zero[8] = {};
    for (int64_t i = c0 + threadIdx.x * 8; i < c1; i += kStep) store8(o + i, c1 - i, zero);
    return;
  }
  __syncthreads();  // every wave has its q
  if (threadIdx.x < 64) {
    const int n = gather_slots(S, K, q, it, c0, c1);
    if (threadIdx.x == 0) n_slots = n;
  }
  // a exp(x - lse), x - lse rounded once; the root of the exponential twice, since the hardware's 2^y has no
  // results below 2^-126 and a may be large
  const auto grad = [&](float v) {
    const float h = pow2(__builtin_fmaf(v, it, -l) * (0.5f * kLog2e));
    return a * h * h;
  };
  int64_t i = lead + at;
  const bool far = !(fabsf(l) < kFarLse);  // (the same for the whole workgroup)
  Norm norm{0.0f, 0.0f, 0.0f};
  if (far) {
    norm = far_row<T, kBwdThreads>(p, V, it * kLog2e, far_part);
    for (int64_t k = c0 + threadIdx.x; k < c1; k += kBwdThreads)
      o[k] = from_f32<T>(a * exp_e(norm.log_p(to_f32(p[k]), it)));
    i = c1;
  } else if (at == 0 && threadIdx.x < lead) {
    o[threadIdx.x] = from_f32<T>(grad(to_f32(p[threadIdx.x])));
  }
  const auto stream = [&](auto unroll) {
    constexpr int U = decltype(unroll)::value;
    for (; i + U * kStep <= c1; i += U * kStep) {
      Raw8<T> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u].load(p + i + u * kStep + threadIdx.x * 8);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[8];
        raw[u].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = grad(v[j]);
        store8_full<PAST>(o + i + u * kStep + threadIdx.x * 8, v);
      }
    }
  };
  stream(Int<kBwdUnroll>{});
  stream(Int<kUnrollRest>{});
  for (; i < c1; i += kStep) {
    float v[8];
    const int64_t k = i + threadIdx.x * 8;
    load8(p + k, c1 - k, 0.0f, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = grad(v[j]);
    store8(o + k, c1 - k, v);
  }
  __syncthreads();  // the piece's stores come before the rewrites
  const int n = n_slots;
  for (int k = threadIdx.x; k < n; k += kBwdThreads) {
    const int32_t v = S.id[k];
    bool first = true;
    float m = 0.0f;  // the q of the word's slots, in slot order
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const bool same = S.id[j] == v;
      first = first && !(same && j < k);
      m += same ? S.t[j] : 0.0f;
    }
    const float lp = far ? norm.log_p(S.x[k], it) : __builtin_fmaf(S.x[k], it, -l);
    if (first) o[v] = from_f32<T>(a * (exp_e(lp) - m));  // the first slot of a repeated word writes it
  }
}

// Workgroups and pieces per row, from the shape alone.
struct Split {
  int n, threads;
  int64_t piece;
};
Split split_into(int64_t V, int64_t n, int64_t step, int threads) {
  const int64_t piece = align_up(ceil_div(V, n < 1 ? 1 : n), step);
  return {static_cast<int>(ceil_div(V, piece)), threads, piece};
}
// Forward: a workgroup per row. 1024 threads when the rows alone leave compute
// units idle, else as many as still make two turns of the main loop (in a step
// at 8192 x 131072 bf16 17 us less with 1024 than with 256, at 4096 x 32768 12 us
// more). A second workgroup for a row costs a second launch and a workspace, 11.5 us
// of wall time at the least, so rows are cut past 2^18 words only. Three float32
// rows in one launch and in two with pieces of 2^14 words, wall time (GPU time):
// 131072 words 8.8 (8.8) and 11.5 us (6.4), 151936 9.9 (9.9) and 11.6 (6.4), 262144
// 13.4 (13.4) and 11.4 (6.4). The pieces of up to 2^18 words taken past the border
// are longer than they need be: 600001 words take 14.7 us (14.5), 12.0 (6.7) with
// pieces of 2^14.
Split fwd_split(int64_t T, int64_t V) {
  const int64_t turn = 8 * kUnroll;
  const int threads = T < 512 || V >= 2 * 1024 * turn ? 1024 : (V >= 2 * 512 * turn ? 512 : 256);
  const int64_t most = ceil_div(V, int64_t(1) << 18), want = T >= 256 || T == 0 ? 1 : ceil_div(512, T);
  return split_into(V, want < most ? want : most, 8192, threads);
}
// Backward: pieces of one turn of the main loop (8192 elements), or of 64
// elements per teacher slot where that is more, since every piece reads the slots.
// The workgroups in flight then cover one stretch of memory, which the memory
// serves faster than a workgroup per row: a step at 4096 x 32768 bf16 takes 137 us
// against 143, at 8192 x 131072 1077 us against 1182 (and 1102 with 1024 threads).
Split bwd_split(int64_t V, int64_t K) {
  const int64_t turn = 8 * kBwdThreads * kBwdUnroll, piece = align_up(64 * K > turn ? 64 * K : turn, turn);
  return {static_cast<int>(ceil_div(V, piece)), kBwdThreads, piece};
}

int check_args(const char* what, int dtype, int t_dtype, int64_t T, int64_t V, int64_t K, double tau) {
  if (int s = check_float_dtype(what, dtype)) return s;
  if (int s = check_float_dtype(what, t_dtype)) return s;
  if (T < 0 || K < 0) return set_error(DET_ERR_INVALID_ARG, "%s: T and K must be >= 0", what);
  if (V < 1) return set_error(DET_ERR_INVALID_ARG, "%s: V must be >= 1", what);
  if (K > kMaxK) return set_error(DET_ERR_UNSUPPORTED, "%s: K must be <= %d, got %lld", what, kMaxK, (long long)K);
  if (V > 0x7FFFFFFF - 65536 || T > 0x7FFFFFFF)
    return set_error(DET_ERR_UNSUPPORTED, "%s: T and V must be < 2^31 - 65536", what);
  if (!(tau >= 1e-6 && tau <= 1e6))
    return set_error(DET_ERR_INVALID_ARG, "%s: tau must lie in [1e-6, 1e6], got %g", what, tau);
  // a launch has at most 2^32 - 1 threads
  if (T * fwd_split(T, V).n > 0xFFFFFFFF / fwd_split(T, V).threads)
    return set_error(DET_ERR_UNSUPPORTED, "%s: problem too large", what);
  if (T * bwd_split(V, K).n > 0xFFFFFFFF / kBwdThreads) return set_error(DET_ERR_UNSUPPORTED, "%s: problem too large", what);
  return DET_OK;
}
int check_ld(const char* what, const char* name, int64_t ld, int64_t n, int64_t T) {
  if (ld < n) return set_error(DET_ERR_INVALID_ARG, "%s: row stride of %s < %lld", what, name, (long long)n);
  if (ld > (int64_t(1) << 44) / T) return set_error(DET_ERR_UNSUPPORTED, "%s: %s is too large", what, name);
  return DET_OK;
}

size_t ws_bytes_for(int64_t T, int64_t V) {
  const Split s = fwd_split(T, V);
  return T == 0 || s.n == 1 ? 0 : DET_WS_HEADER_BYTES + align_up(static_cast<size_t>(T * s.n) * sizeof(MaxSum), 256);
}

template <typename T, typename TT>
void launch_fwd(const void* z, int64_t ld, int64_t V, const int32_t* ids, int64_t ids_ld, const void* t, int64_t t_ld,
                int64_t rows, int64_t K, float it, float* loss, float* lse, MaxSum* slots, hipStream_t st) {
  const Split s = fwd_split(rows, V);
  const dim3 grid(static_cast<uint32_t>(rows * s.n));
#define DET_DISTILL_FWD(THREADS)                                                                                      \
  hipLaunchKernelGGL((distill_fwd_kernel<T, TT, THREADS>), grid, dim3(THREADS), 0, st, static_cast<const T*>(z), ld, V, \
                     ids, ids_ld, static_cast<const TT*>(t), t_ld, (int)K, it, s.n, s.piece, slots, loss, lse)
  if (s.threads == 256) DET_DISTILL_FWD(256);
  else if (s.threads == 512) DET_DISTILL_FWD(512);
  else DET_DISTILL_FWD(1024);
#undef DET_DISTILL_FWD
  if (s.n > 1)
    hipLaunchKernelGGL((distill_join_kernel<T, TT>), dim3(static_cast<uint32_t>(rows)), dim3(256), 0, st,
                       static_cast<const T*>(z), ld, V, ids, ids_ld, static_cast<const TT*>(t), t_ld, (int)K, it, s.n,
                       slots, loss, lse);
}
template <typename T, typename TT>
void launch_bwd(void* dz, int64_t ld_d, const void* z, int64_t ld, int64_t V, const int32_t* ids, int64_t ids_ld,
                const void* t, int64_t t_ld, int64_t rows, int64_t K, float it, const float* lse, const float* dloss,
                hipStream_t st) {
  const Split s = bwd_split(V, K);
  const dim3 grid(static_cast<uint32_t>(rows * s.n));
#define DET_DISTILL_BWD(PAST)                                                                                        \
  hipLaunchKernelGGL((distill_bwd_kernel<T, TT, PAST>), grid, dim3(kBwdThreads), 0, st, static_cast<T*>(dz), ld_d,   \
                     static_cast<const T*>(z), ld, V, ids, ids_ld, static_cast<const TT*>(t), t_ld, (int)K, it, s.n, \
                     s.piece, lse, dloss)
  if (past_caches(rows * V * static_cast<int64_t>(sizeof(T)))) DET_DISTILL_BWD(true);
  else DET_DISTILL_BWD(false);
#undef DET_DISTILL_BWD
}

}  // namespace
}  // namespace detgrad

using namespace detgrad;

#define DET_DISTILL_BY_TYPE(F, ...)                                                              \
  if (dtype == DET_BF16) {                                                                       \
    if (teacher_dtype == DET_BF16) F<uint16_t, uint16_t>(__VA_ARGS__);                           \
    else F<uint16_t, float>(__VA_ARGS__);                                                        \
  } else {                                                                                       \
    if (teacher_dtype == DET_BF16) F<float, uint16_t>(__VA_ARGS__);                              \
    else F<float, float>(__VA_ARGS__);                                                           \
  }

extern "C" int det_topk_distill_workspace_size(int64_t T, int64_t V, int64_t K, size_t* bytes) {
  if (!bytes) return set_error(DET_ERR_INVALID_ARG, "topk_distill: bytes is NULL");
  if (int s = check_args("topk_distill", DET_BF16, DET_BF16, T, V, K, 1.0)) return s;
  *bytes = ws_bytes_for(T, V);
  return ok();
}

extern "C" int det_topk_distill(const void* logits, int64_t ld, int dtype, const int32_t* ids, int64_t ids_ld,
                                const void* teacher, int64_t teacher_ld, int teacher_dtype, int64_t T, int64_t V,
                                int64_t K, double tau, float* loss, float* lse, void* ws, size_t ws_bytes,
                                void* stream) {
  const char* what = "topk_distill";
  if (int s = check_args(what, dtype, teacher_dtype, T, V, K, tau)) return s;
  if (T == 0) return ok();
  if (!logits || !loss || !lse || (K && (!ids || !teacher)))
    return set_error(DET_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if (int s = check_ld(what, "logits", ld, V, T)) return s;
  if (int s = check_ld(what, "ids", ids_ld, K, T)) return s;
  if (int s = check_ld(what, "teacher", teacher_ld, K, T)) return s;
  const size_t need = ws_bytes_for(T, V);
  if (int s = check_workspace(ws, ws_bytes, need)) return s;
  const size_t es = dtype_size(dtype), ts = dtype_size(teacher_dtype);
  const Buf outs[] = {{"loss", range1d(loss, T * 4)},
                      {"lse", range1d(lse, T * 4)},
                      {"the workspace", range1d(need ? ws : nullptr, ws_bytes)}};
  const Buf ins[] = {buf_rows("logits", logits, T, V, ld, es),
                     buf_rows("ids", ids, T, K, ids_ld, 4),
                     buf_rows("teacher", teacher, T, K, teacher_ld, ts)};
  if (int s = check_buffers(what, outs, 3, ins, 3)) return s;
  auto* slots = need ? reinterpret_cast<MaxSum*>(static_cast<char*>(ws) + DET_WS_HEADER_BYTES) : nullptr;
  const float it = static_cast<float>(1.0 / tau);
  DET_DISTILL_BY_TYPE(launch_fwd, logits, ld, V, ids, ids_ld, teacher, teacher_ld, T, K, it, loss, lse, slots,
                      as_stream(stream))
  return check_launch("det_topk_distill");
}

extern "C" int det_topk_distill_bwd(void* dlogits, int64_t ld_d, const void* logits, int64_t ld, int dtype,
                                    const int32_t* ids, int64_t ids_ld, const void* teacher, int64_t teacher_ld,
                                    int teacher_dtype, int64_t T, int64_t V, int64_t K, double tau, const float* lse,
                                    const float* dloss, void* stream) {
  const char* what = "topk_distill_bwd";
  if (int s = check_args(what, dtype, teacher_dtype, T, V, K, tau)) return s;
  if (T == 0) return ok();
  if (!dlogits || !logits || !lse || !dloss || (K && (!ids || !teacher)))
    return set_error(DET_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if (int s = check_ld(what, "dlogits", ld_d, V, T)) return s;
  if (int s = check_ld(what, "logits", ld, V, T)) return s;
  if (int s = check_ld(what, "ids", ids_ld, K, T)) return s;
  if (int s = check_ld(what, "teacher", teacher_ld, K, T)) return s;
  const size_t es = dtype_size(dtype), ts = dtype_size(teacher_dtype);
  const Buf outs[] = {buf_rows("dlogits", dlogits, T, V, ld_d, es)};
  const Buf ins[] = {buf_rows("logits", logits, T, V, ld, es),
                     buf_rows("ids", ids, T, K, ids_ld, 4),
                     buf_rows("teacher", teacher, T, K, teacher_ld, ts),
                     {"lse", range1d(lse, T * 4)},
                     {"dloss", range1d(dloss, T * 4)}};
  if (int s = check_buffers(what, outs, 1, ins, 5)) return s;
  const float it = static_cast<float>(1.0 / tau);
  DET_DISTILL_BY_TYPE(launch_bwd, dlogits, ld_d, logits, ld, V, ids, ids_ld, teacher, teacher_ld, T, K, it, lse, dloss,
                      as_stream(stream))
  return check_launch("det_topk_distill_bwd");
}
