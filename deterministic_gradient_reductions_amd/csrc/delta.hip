// det_delta_rule: the gated delta rule over packed sequences, in chunks.
//
//   S' = exp(g_t) S_{t-1},  u_t = beta_t (v_t - S'^T k_t),  S_t = S' + k_t u_t^T,  o_t = scale S_t^T q_t
//
// A chunk of C tokens from the state S0 on, with G the running sum of g inside it,
// D_ij = exp(G_i - G_j) for j <= i, M = D * K K^T below the diagonal, P = scale D * Q K^T
// up to it, B = diag(beta):
//
//   N = (I + M B)^-1 (V - e^G K S0),  U = B N
//   O = scale e^G Q S0 + P U,         S1 = e^G_C S0 + K^T (e^(G_C - G) U)
//
// No exponent above is positive where g is not, however strong the decays, so
// nothing is divided by a small decay; differences of G keep the digits that a
// float32 sum over a chunk would lose (two words). g below -1e4 counts as -1e4 (a
// factor of 0 either way), which keeps -inf out of the differences.
//
// Two kernels. The first, all chunks side by side, inverts I + M B (a wave per
// chunk and head: 16 x 16 diagonal blocks by substitution, the blocks below by
// float32 matrix instructions). The second walks the chunks of one sequence and
// value head in order; a wave owns 16 columns of v, so its part of S, R, N, U and O
// depends on no other wave, and what one product leaves in its registers is the next
// one's operand. The waves of a workgroup share the fragments of K, Q, K^T, the
// inverse and P in LDS.
#include "delta.hpp"

namespace detgrad {
namespace {

// exp(hi + lo) of a difference of two-word sums
__device__ __forceinline__ float decay(float hi_i, float lo_i, float hi_j, float lo_j) {
  return exp_e((hi_i - hi_j) + (lo_i - lo_j));
}

constexpr int kPrepWaves = 4;

template <typename T, int DK>
__global__ __launch_bounds__(64 * kPrepWaves) void delta_prep_kernel(DeltaSizes z, Heads<const T> k,
                                                                     const float* __restrict__ g, int64_t g_ld,
                                                                     const T* __restrict__ beta, int64_t beta_ld,
                                                                     float* __restrict__ inverse, float* __restrict__ gates,
                                                                     int64_t units) {
  constexpr int kIn = DeltaType<T>::kIn, kLogC = DeltaType<T>::kLogC, C = 1 << kLogC, RT = C / 16, KS = DK / 32;
  constexpr int kLd = C + 4;  // 16-byte rows whose starts move through the banks
  __shared__ float lds[kPrepWaves][C * kLd + 3 * C];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, lg = lane >> 4;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kPrepWaves + wave;
  if (unit >= units) return;
  const uint32_t tile = static_cast<uint32_t>(unit / z.H);
  const int h = static_cast<int>(unit % z.H), hk = h / (z.H / z.Hk);
  int e;
  uint32_t r0, r1, s0, s1;
  if (!segment_tile<1>(z.offs, z.S, static_cast<uint32_t>(z.T), kLogC, tile, e, r0, r1, s0, s1)) return;
  const int n = static_cast<int>(r1 - r0);
  float* a = lds[wave];
  float *hi = a + C * kLd, *lo = hi + C, *be = lo + C;

  // the sums of g in float64, kept as two float32 words
  {
    double G = 0.0;
    float b = 0.0f;
    if (lane < n) {
      const float x = g[(r0 + lane) * g_ld + h];
      G = x < -1e4f ? -1e4f : x;
      b = to_f32(beta[(r0 + lane) * beta_ld + h]);
    }
#pragma unroll
    for (int d = 1; d < C; d <<= 1) {
      const double o = __shfl_up(G, d);
      if (lane >= d) G += o;
    }
    const double last = __shfl(G, C - 1);
    const float h0 = static_cast<float>(G), h1 = static_cast<float>(G - h0);
    float* out = gates + unit * (kGateRows * C);
    if (lane < C) {
      hi[lane] = h0;
      lo[lane] = h1;
      be[lane] = b;
      out[kGHi * C + lane] = h0;
      out[kGLo * C + lane] = h1;
      out[kEG * C + lane] = exp_e(h0) * (1.0f + h1);
      const double rest = last - G;
      const float q0 = static_cast<float>(rest);
      out[kRest * C + lane] = exp_e(q0) * (1.0f + static_cast<float>(rest - q0));
      out[kBeta * C + lane] = b;
    }
  }
  wave_fence();

  // K K^T: fragments straight from memory, eight channels 32 ks + 8 lg .. in a lane
  f32x4 kk[RT][RT] = {};
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    Frag<kIn> f[RT];
    const int d = 32 * ks + 8 * lg;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int t = 16 * rt + c;
      float v[8] = {};
      if (t < n && d < z.dk) load8(k.row(r0 + t, hk) + d, z.dk - d, 0.0f, v);
      f[rt] = frag_of<kIn>(f32x4{v[0], v[1], v[2], v[3]}, f32x4{v[4], v[5], v[6], v[7]});
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j <= i; ++j) mm<kIn>(kk[i][j], f[i], f[j]);
  }
  // M B into LDS, rows i, columns j < i
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j <= i; ++j) {
      const int col = 16 * j + c;
      const float hj = hi[col], lj = lo[col], bj = be[col];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * lg + r;
        a[row * kLd + col] = col < row ? kk[i][j][r] * decay(hi[row], lo[row], hj, lj) * bj : 0.0f;
      }
    }
  wave_fence();

  // The inverses of the diagonal blocks: lane group lg takes block lg, lane c its
  // column c, by substitution down the rows.
  float x[16];
  {
    const int blk = lg < RT ? lg : 0;
    const float* p = a + (16 * blk) * kLd + 16 * blk;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float s = r == c ? 1.0f : 0.0f;
#pragma unroll
      for (int m = 0; m < r; m += 4) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(p + r * kLd + m);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (m + q < r) s = __builtin_fmaf(-w[q], x[m + q], s);
      }
      x[r] = s;
    }
    wave_fence();
    if (lg < RT)
#pragma unroll
      for (int r = 0; r < 16; ++r) a[(16 * blk + r) * kLd + 16 * blk + c] = x[r];
  }
  wave_fence();

  // The blocks below, column by column of blocks: X_ij = -X_ii sum_{j <= m < i} (M B)_im X_mj.
  // Float32 matrix instructions; the place 4 lg + s of the sum is step s of lane group lg.
  const auto row4 = [&](int i, int j) { return *reinterpret_cast<const f32x4*>(a + (16 * i + c) * kLd + 16 * j + 4 * lg); };
  float* out = inverse + unit * (C * C);
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    f32x4 X[RT];
#pragma unroll
    for (int r = 0; r < 4; ++r) X[j][r] = a[(16 * j + 4 * lg + r) * kLd + 16 * j + c];
#pragma unroll
    for (int i = j + 1; i < RT; ++i) {
      f32x4 w{}, y{};
#pragma unroll
      for (int m = j; m < i; ++m) {
        const f32x4 u = row4(i, m);
#pragma unroll
        for (int s = 0; s < 4; ++s) w = __builtin_amdgcn_mfma_f32_16x16x4f32(u[s], X[m][s], w, 0, 0, 0);
      }
      const f32x4 u = row4(i, i);
#pragma unroll
      for (int s = 0; s < 4; ++s) y = __builtin_amdgcn_mfma_f32_16x16x4f32(-u[s], w[s], y, 0, 0, 0);
      X[i] = y;
    }
#pragma unroll
    for (int i = j; i < RT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) out[(16 * i + 4 * lg + r) * C + 16 * j + c] = X[i][r];
  }
}

// What the chunk kernel takes and gives.
template <typename T>
struct FwdArgs {
  Heads<const T> q, k, v;
  Heads<T> o;
  const float *inverse, *gates, *s0;
  float *s1, *states;
};

// Workgroup (x, s): value head x / n_blocks, columns 16 NW (x % n_blocks) .. of sequence s.
template <typename T, int DK, int NW>
__global__ __launch_bounds__(64 * NW) void delta_fwd_kernel(DeltaSizes z, FwdArgs<T> A, int n_blocks) {
  constexpr int kIn = DeltaType<T>::kIn, kOut = DeltaType<T>::kOut, kLogC = DeltaType<T>::kLogC, C = 1 << kLogC;
  constexpr int RT = C / 16, KC = C / 32, DT = DK / 16, KD = DK / 32, kW = kStateWords;
  using RowImg = Image<RT, KD, kIn>;   // rows t, places d
  using ColImg = Image<DT, KC, kIn>;   // rows d, places t
  using InvImg = Image<RT, KC, kW>;    // rows i, places j
  using PImg = Image<RT, KC, kOut>;    // rows i, places j
  constexpr int kK = 0, kQ = kK + RowImg::kBytes, kKT = kQ + RowImg::kBytes, kInv = kKT + ColImg::kBytes,
                kP = kInv + InvImg::kBytes, kG = kP + PImg::kBytes, kAll = kG + kGateRows * C * 4;
  __shared__ __align__(16) char lds[kAll];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, lg = lane >> 4;
  const int h = blockIdx.x / n_blocks, hk = h / (z.H / z.Hk), v0 = ((blockIdx.x % n_blocks) * NW + wave) * 16;
  const int s = blockIdx.y;
  const float* gate = reinterpret_cast<const float*>(lds + kG);
  uint32_t r0, r1, first;
  segment_rows(z.offs, s, static_cast<uint32_t>(z.T), kLogC, r0, r1, first);

  // tiles of the images above the diagonal stay zero
  for (int i = threadIdx.x * 16; i < kG - kInv; i += 64 * NW * 16) *reinterpret_cast<u32x4*>(lds + kInv + i) = u32x4{0, 0, 0, 0};

  // the state's rows 16 i + 4 lg + r, column v0 + c
  const int col = v0 + c;
  const bool live = col < z.dv;
  const int64_t size = static_cast<int64_t>(z.dk) * z.dv, of = (static_cast<int64_t>(s) * z.H + h) * size;
  f32x4 S[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = 16 * i + 4 * lg + r;
      S[i][r] = A.s0 && live && d < z.dk ? A.s0[of + static_cast<int64_t>(d) * z.dv + col] : 0.0f;
    }
  const auto write_state = [&](float* p) {
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = 16 * i + 4 * lg + r;
        if (live && d < z.dk) p[static_cast<int64_t>(d) * z.dv + col] = S[i][r];
      }
  };

  // What a thread brings from memory for a chunk: blocks of four tokens by four channels
  // of K and Q, of four by four of the inverse, gates, and its own elements of V.
  constexpr int kThreads = 64 * NW, kRowBlocks = C * DK / 16, kInvBlocks = C * C / 16;
  constexpr int kNB = (kRowBlocks + kThreads - 1) / kThreads, kNI = (kInvBlocks + kThreads - 1) / kThreads;
  constexpr int kNG = (kGateRows * C + kThreads - 1) / kThreads;
  Raw4<T> rk[kNB][4], rq[kNB][4];
  f32x4 ri[kNI][4];
  float rg[kNG];
  T rv[RT][4];
  const auto fetch = [&](uint32_t t0, int64_t unit) {
    const int n = r1 - t0 < static_cast<uint32_t>(C) ? static_cast<int>(r1 - t0) : C;
#pragma unroll
    for (int b = 0; b < kNB; ++b) {
      const int id = b * kThreads + threadIdx.x, t = id / (DK / 4) * 4, d = id % (DK / 4) * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = id < kRowBlocks && t + j < n ? z.dk - d : 0;
        const int64_t row = m > 0 ? t0 + t + j : t0;
        rk[b][j].load(A.k.row(row, hk) + d, m);
        rq[b][j].load(A.q.row(row, hk) + d, m);
      }
    }
    const float* inv = A.inverse + unit * (C * C);
#pragma unroll
    for (int b = 0; b < kNI; ++b) {
      const int id = b * kThreads + threadIdx.x, i = id / (C / 4) * 4, j = id % (C / 4) * 4;
      if (id < kInvBlocks && j / 16 <= i / 16)
#pragma unroll
        for (int r = 0; r < 4; ++r) ri[b][r] = *reinterpret_cast<const f32x4*>(inv + (i + r) * C + j);
    }
#pragma unroll
    for (int b = 0; b < kNG; ++b) {
      const int id = b * kThreads + threadIdx.x;
      if (id < kGateRows * C) rg[b] = A.gates[unit * (kGateRows * C) + id];
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * i + 4 * lg + r;
        rv[i][r] = live && t < n ? A.v.row(t0 + t, h)[col] : T{};
      }
  };

  int64_t unit = static_cast<int64_t>(first) * z.H + h;
  if (r0 < r1) fetch(r0, unit);
  for (uint32_t t0 = r0; t0 < r1; t0 += C, unit += z.H) {
    const int n = r1 - t0 < static_cast<uint32_t>(C) ? static_cast<int>(r1 - t0) : C;
    __syncthreads();  // the last chunk's fragments have been read
#pragma unroll
    for (int b = 0; b < kNB; ++b) {
      const int id = b * kThreads + threadIdx.x, t = id / (DK / 4) * 4, d = id % (DK / 4) * 4;
      if (id < kRowBlocks) {
        float x[4][4], y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          rk[b][j].get(x[j]);
          RowImg::store4(lds + kK, t + j, d, x[j]);
          rq[b][j].get(y);
          RowImg::store4(lds + kQ, t + j, d, y);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float w[4] = {x[0][j], x[1][j], x[2][j], x[3][j]};
          ColImg::store4(lds + kKT, d + j, t, w);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kNI; ++b) {
      const int id = b * kThreads + threadIdx.x, i = id / (C / 4) * 4, j = id % (C / 4) * 4;
      if (id < kInvBlocks && j / 16 <= i / 16)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float w[4] = {ri[b][r][0], ri[b][r][1], ri[b][r][2], ri[b][r][3]};
          InvImg::store4(lds + kInv, i + r, j, w);
        }
    }
#pragma unroll
    for (int b = 0; b < kNG; ++b) {
      const int id = b * kThreads + threadIdx.x;
      if (id < kGateRows * C) reinterpret_cast<float*>(lds + kG)[id] = rg[b];
    }
    f32x4 R[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) R[i][r] = to_f32(rv[i][r]);
    __syncthreads();
    if (t0 + C < r1) fetch(t0 + C, unit + z.H);
    if (A.states) write_state(A.states + unit * size);

    // P, its tiles shared out among the waves: rows j of the result are places of the image
    for (int p = wave; p < RT * (RT + 1) / 2; p += NW) {
      int i = 0, j = p;
      while (j > i) j -= ++i;
      f32x4 acc{};
#pragma unroll
      for (int ks = 0; ks < KD; ++ks)
        mm<kIn>(acc, RowImg::load(lds + kK, j, ks), RowImg::load(lds + kQ, i, ks));
      const int row = 16 * i + c;
      float w[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = 16 * j + 4 * lg + r;
        const float dcy = decay(gate[kGHi * C + row], gate[kGLo * C + row], gate[kGHi * C + m], gate[kGLo * C + m]);
        w[r] = m <= row ? acc[r] * dcy * z.scale : 0.0f;
      }
      PImg::store4(lds + kP, row, 16 * j + 4 * lg, w);
    }
    // K S0 (rows t, columns v) and its transposed Q S0 (rows v, columns t)
    f32x4 ks0[RT] = {}, o[RT] = {};
#pragma unroll
    for (int ks = 0; ks < KD; ++ks) {
      const Frag<kW> f = frag_of<kW>(S[2 * ks], S[2 * ks + 1]);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        mm<kW>(ks0[i], RowImg::load(lds + kK, i, ks), f);
        mm<kOut>(o[i], f, RowImg::load(lds + kQ, i, ks));
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const f32x4 eg = *reinterpret_cast<const f32x4*>(gate + kEG * C + 16 * i + 4 * lg);
      const float e_col = gate[kEG * C + 16 * i + c] * z.scale;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        R[i][r] = __builtin_fmaf(-eg[r], ks0[i][r], R[i][r]);
        o[i][r] *= e_col;
      }
    }
    // N, then U = beta N
    f32x4 U[RT] = {};
#pragma unroll
    for (int kt = 0; kt < KC; ++kt) {
      const Frag<kW> f = frag_of<kW>(R[2 * kt], R[2 * kt + 1]);
#pragma unroll
      for (int i = 2 * kt; i < RT; ++i) mm<kW>(U[i], InvImg::load(lds + kInv, i, kt), f);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) U[i] *= *reinterpret_cast<const f32x4*>(gate + kBeta * C + 16 * i + 4 * lg);
    __syncthreads();  // P is there
#pragma unroll
    for (int kt = 0; kt < KC; ++kt) {
      const Frag<kOut> f = frag_of<kOut>(U[2 * kt], U[2 * kt + 1]);
#pragma unroll
      for (int i = 2 * kt; i < RT; ++i) mm<kOut>(o[i], f, PImg::load(lds + kP, i, kt));
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int t = 16 * i + c;
      if (t < n) store4(A.o.row(t0 + t, h) + v0 + 4 * lg, z.dv - v0 - 4 * lg, o[i]);
    }
    // S1
    const float el = gate[kEG * C + C - 1];
#pragma unroll
    for (int i = 0; i < DT; ++i) S[i] *= el;
#pragma unroll
    for (int kt = 0; kt < KC; ++kt) {
      const f32x4 w0 = *reinterpret_cast<const f32x4*>(gate + kRest * C + 32 * kt + 4 * lg);
      const f32x4 w1 = *reinterpret_cast<const f32x4*>(gate + kRest * C + 32 * kt + 16 + 4 * lg);
      const Frag<kW> f = frag_of<kW>(U[2 * kt] * w0, U[2 * kt + 1] * w1);
#pragma unroll
      for (int i = 0; i < DT; ++i) mm<kW>(S[i], ColImg::load(lds + kKT, i, kt), f);
    }
  }
  if (A.s1) write_state(A.s1 + of);
}

struct Layout {
  size_t inverse, gates, all;
};
Layout layout_of(const DeltaSizes& z, int dtype) {
  const int64_t C = dtype == DET_BF16 ? 64 : 32, units = delta_tiles(z.T, z.S, dtype) * z.H;
  Layout l;
  l.inverse = DET_WS_HEADER_BYTES;
  l.gates = l.inverse + static_cast<size_t>(units * C * C) * 4;
  l.all = l.gates + align_up(static_cast<size_t>(units * kGateRows * C) * 4, 256);
  return l;
}

template <typename T, int DK>
void launch_prep(const DeltaSizes& z, const void* k, int64_t k_st, int64_t k_sh, const float* g, int64_t g_ld,
                 const void* beta, int64_t beta_ld, float* inverse, float* gates, int64_t units, hipStream_t st) {
  hipLaunchKernelGGL((delta_prep_kernel<T, DK>), dim3(static_cast<uint32_t>(ceil_div(units, kPrepWaves))),
                     dim3(64 * kPrepWaves), 0, st, z, Heads<const T>{static_cast<const T*>(k), k_st, k_sh}, g, g_ld,
                     static_cast<const T*>(beta), beta_ld, inverse, gates, units);
}

template <typename T, int DK>
void launch_fwd(const DeltaSizes& z, const FwdArgs<T>& A, hipStream_t st) {
  // the widest workgroup that still leaves one for each compute unit
  int nw = 8;
  while (nw > 1 && (static_cast<int64_t>(z.S) * z.H * ceil_div(z.dv, 16 * nw) < 256 || 16 * nw >= 2 * z.dv)) nw /= 2;
  const int n_blocks = static_cast<int>(ceil_div(z.dv, 16 * nw));
  const dim3 grid(static_cast<uint32_t>(z.H * n_blocks), static_cast<uint32_t>(z.S));
#define DET_DELTA_FWD(NW) \
  case NW: hipLaunchKernelGGL((delta_fwd_kernel<T, DK, NW>), grid, dim3(64 * NW), 0, st, z, A, n_blocks); break;
  switch (nw) {
    DET_DELTA_FWD(1)
    DET_DELTA_FWD(2)
    DET_DELTA_FWD(4)
    DET_DELTA_FWD(8)
  }
#undef DET_DELTA_FWD
}

}  // namespace

void delta_prepare(const DeltaSizes& z, int dtype, const void* k, int64_t k_st, int64_t k_sh, const float* g, int64_t g_ld,
                   const void* beta, int64_t beta_ld, float* inverse, float* gates, hipStream_t st) {
  const int64_t units = delta_tiles(z.T, z.S, dtype) * z.H;
#define DET_DELTA_PREP(T, DK) launch_prep<T, DK>(z, k, k_st, k_sh, g, g_ld, beta, beta_ld, inverse, gates, units, st)
  if (dtype == DET_BF16) {
    if (z.dk <= 64) DET_DELTA_PREP(uint16_t, 64);
    else DET_DELTA_PREP(uint16_t, 128);
  } else {
    if (z.dk <= 64) DET_DELTA_PREP(float, 64);
    else DET_DELTA_PREP(float, 128);
  }
#undef DET_DELTA_PREP
}

int delta_check_sizes(const char* what, int dtype, int64_t T, int64_t S, int64_t Hk, int64_t H, int64_t dk, int64_t dv) {
  if (int s = check_float_dtype(what, dtype)) return s;
  if (T < 0 || S < 0) return set_error(DET_ERR_INVALID_ARG, "%s: T and S must be >= 0", what);
  if (Hk < 1 || H < 1 || H % Hk)
    return set_error(DET_ERR_INVALID_ARG, "%s: the value heads must be a multiple of the key heads", what);
  if (dk < 1 || dv < 1) return set_error(DET_ERR_INVALID_ARG, "%s: head sizes must be >= 1", what);
  if (dk > kDeltaMaxDim || dv > kDeltaMaxDim)
    return set_error(DET_ERR_UNSUPPORTED, "%s: head sizes must be <= %d, got %lld and %lld", what, kDeltaMaxDim,
                     (long long)dk, (long long)dv);
  if (S > 65535) return set_error(DET_ERR_UNSUPPORTED, "%s: S must be <= 65535", what);
  if (T >= (int64_t(1) << 31) - 65536 || H > 65535 || (delta_tiles(T, S, dtype) + 1) * H >= (int64_t(1) << 23))  // 512 threads for each at most
    return set_error(DET_ERR_UNSUPPORTED, "%s: problem too large", what);
  return DET_OK;
}

int delta_buf(const char* what, const char* name, const void* p, int64_t T, int64_t heads, int64_t dim, int64_t st, int64_t sh,
              size_t elem, Buf& out) {
  out = Buf{name, Range{}, elem, 0, 0};
  if (!p || T == 0 || heads == 0) return DET_OK;
  // one token, one head: that stride is not used
  const bool by_token = (heads == 1 || sh >= dim) && (T == 1 || st >= (heads - 1) * sh + dim);
  const bool by_head = (T == 1 || st >= dim) && (heads == 1 || sh >= (T - 1) * st + dim);
  if (!by_token && !by_head)
    return set_error(DET_ERR_INVALID_ARG, "%s: strides of %s overlap (token %lld, head %lld)", what, name, (long long)st,
                     (long long)sh);
  const int64_t most = (int64_t(1) << 44);
  if (st > most / T || sh > most / heads) return set_error(DET_ERR_UNSUPPORTED, "%s: %s is too large", what, name);
  if (by_token) out = buf_rows(name, p, T, (heads - 1) * (heads > 1 ? sh : 0) + dim, T > 1 ? st : (heads - 1) * sh + dim, elem);
  else out = buf_rows(name, p, heads, (T - 1) * (T > 1 ? st : 0) + dim, sh, elem);
  return DET_OK;
}

}  // namespace detgrad

using namespace detgrad;

extern "C" int det_delta_rule_chunks(int64_t T, int64_t S, int dtype, int64_t* chunks) {
  if (!chunks) return set_error(DET_ERR_INVALID_ARG, "delta_rule: chunks is NULL");
  if (int s = delta_check_sizes("delta_rule", dtype, T, S, 1, 1, 1, 1)) return s;
  *chunks = delta_tiles(T, S, dtype);
  return ok();
}

extern "C" int det_delta_rule_workspace_size(int64_t T, int64_t S, int64_t H, int dtype, size_t* bytes) {
  if (!bytes) return set_error(DET_ERR_INVALID_ARG, "delta_rule: bytes is NULL");
  if (int s = delta_check_sizes("delta_rule", dtype, T, S, 1, H, 1, 1)) return s;
  DeltaSizes z{};
  z.T = T;
  z.S = static_cast<int>(S);
  z.H = static_cast<int>(H);
  *bytes = T == 0 ? 0 : layout_of(z, dtype).all;
  return ok();
}

extern "C" int det_delta_rule(const void* q, int64_t q_st, int64_t q_sh, const void* k, int64_t k_st, int64_t k_sh,
                              const void* v, int64_t v_st, int64_t v_sh, const float* g, int64_t g_ld, const void* beta,
                              int64_t beta_ld, int dtype, int64_t T, int64_t Hk, int64_t H, int64_t dk, int64_t dv,
                              const int32_t* offs, int64_t S, double scale, const float* initial_state, void* o,
                              int64_t o_st, int64_t o_sh, float* final_state, float* states, void* ws, size_t ws_bytes,
                              void* stream) {
  const char* what = "delta_rule";
  if (int s = delta_check_sizes(what, dtype, T, S, Hk, H, dk, dv)) return s;
  if (!(scale > -1e30 && scale < 1e30)) return set_error(DET_ERR_INVALID_ARG, "%s: scale must be finite", what);
  if (S == 0) return ok();
  if (!offs || (T > 0 && (!q || !k || !v || !g || !beta || !o)))
    return set_error(DET_ERR_INVALID_ARG, "%s: NULL pointer", what);
  const size_t es = dtype_size(dtype);
  Buf bq, bk, bv, bo;
  if (int s = delta_buf(what, "q", q, T, Hk, dk, q_st, q_sh, es, bq)) return s;
  if (int s = delta_buf(what, "k", k, T, Hk, dk, k_st, k_sh, es, bk)) return s;
  if (int s = delta_buf(what, "v", v, T, H, dv, v_st, v_sh, es, bv)) return s;
  if (int s = delta_buf(what, "o", o, T, H, dv, o_st, o_sh, es, bo)) return s;
  if (T > 1 && (g_ld < H || beta_ld < H)) return set_error(DET_ERR_INVALID_ARG, "%s: row stride of g or beta < H", what);
  if (T > 0 && (g_ld > (int64_t(1) << 44) / T || beta_ld > (int64_t(1) << 44) / T))
    return set_error(DET_ERR_UNSUPPORTED, "%s: g or beta is too large", what);
  const DeltaSizes z{T, (int)S, (int)Hk, (int)H, (int)dk, (int)dv, offs, static_cast<float>(scale)};
  const Layout l = layout_of(z, dtype);
  const size_t need = T ? l.all : 0;
  if (int s = check_workspace(ws, ws_bytes, need)) return s;
  const size_t state = static_cast<size_t>(H * dk * dv) * 4;
  const Buf outs[] = {bo,
                      {"final_state", range1d(final_state, S * state)},
                      {"states", range1d(states, delta_tiles(T, S, dtype) * state)},
                      {"the workspace", range1d(need ? ws : nullptr, ws_bytes)}};
  const Buf ins[] = {bq, bk, bv, buf_rows("g", g, T, H, T > 1 ? g_ld : H, 4),
                     buf_rows("beta", beta, T, H, T > 1 ? beta_ld : H, es),
                     {"offs", range1d(offs, (S + 1) * 4)},
                     {"initial_state", range1d(initial_state, S * state)}};
  if (int s = check_buffers(what, outs, 4, ins, 7)) return s;
  const hipStream_t st = as_stream(stream);
  float *inverse = nullptr, *gates = nullptr;
  if (T) {
    inverse = reinterpret_cast<float*>(static_cast<char*>(ws) + l.inverse);
    gates = reinterpret_cast<float*>(static_cast<char*>(ws) + l.gates);
    delta_prepare(z, dtype, k, k_st, k_sh, g, g_ld, beta, beta_ld, inverse, gates, st);
  }
#define DET_DELTA_FWD(E)                                                                                             \
  {                                                                                                                  \
    const FwdArgs<E> A{{static_cast<const E*>(q), q_st, q_sh}, {static_cast<const E*>(k), k_st, k_sh},               \
                       {static_cast<const E*>(v), v_st, v_sh}, {static_cast<E*>(o), o_st, o_sh},                     \
                       inverse, gates, initial_state, final_state, states};                                          \
    if (dk <= 64) launch_fwd<E, 64>(z, A, st);                                                                       \
    else launch_fwd<E, 128>(z, A, st);                                                                               \
  }
  if (dtype == DET_BF16) DET_DELTA_FWD(uint16_t)
  else DET_DELTA_FWD(float)
#undef DET_DELTA_FWD
  return check_launch("det_delta_rule");
}
