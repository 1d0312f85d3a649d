// det_delta_rule_bwd: the gradients of the gated delta rule, in the chunks and with the
// notation of its forward. With X = strict(dN N^T), dP = lower(dO U^T) and dS1 the
// gradient of the state behind the chunk:
//
//   dU = P^T dO + e^(G_C - G) K dS1,   dN = (I + M B)^-T B dU,   dV = dN
//   dS0 = e^G_C dS1 + scale (e^G Q)^T dO - (e^G K)^T dN
//   dQ = scale e^G dO S0^T + scale (dP * D) K
//   dK = e^(G_C - G) U dS1^T - e^G dN S0^T + scale (dP * D)^T Q + (Z + Z^T) K,   Z = -D * X * beta_col
//   dbeta = rowsum(dU * N) - colsum(M * X)
//   dG = rowsum(E) - colsum(E) + rowsum(dO * scale e^G Q S0) - rowsum(dN * e^G K S0) - w,   E = dP * P - M * X * beta_col
//        and on the chunk's last row sum(w) + e^G_C <S0, dS1>,   w = rowsum(U * e^(G_C - G) K dS1)
//   dg = the sums of dG from a row to the chunk's end
//
// Nothing is divided by beta or by a decay. Three kernels: the forward's first (the
// inverses), one that walks a sequence's chunks backwards as the forward's second walks
// them (16 columns of v per wave, dS in registers; it writes dV and every chunk's
// dS1), and one for all chunks side by side that forms N, dU and dN of its chunk again
// and the sums over v and over token pairs. In that one a wave owns 16 columns of v
// first (N, dN), then tiles of token pairs, then 16 channels of dQ and dK; N, dN and the
// pair matrices change hands in LDS.
#include "delta.hpp"

namespace detgrad {
namespace {

__device__ __forceinline__ float decay(float hi_i, float lo_i, float hi_j, float lo_j) {
  return exp_e((hi_i - hi_j) + (lo_i - lo_j));
}
__device__ __forceinline__ f32x4 gate4(const float* gate, int C, int row, int at) {
  return *reinterpret_cast<const f32x4*>(gate + row * C + at);
}

// The fragment of places 32 ks .. of a row in memory (n elements from p on, zeros behind them).
template <int NP, typename T>
__device__ __forceinline__ Frag<NP> row_frag(const T* p, int n, int ks) {
  const int at = 32 * ks + 4 * ((threadIdx.x & 63) >> 4);
  Raw4<T> a, b;
  a.load(p + (n > at ? at : 0), n - at);
  b.load(p + (n > at + 16 ? at + 16 : 0), n - at - 16);
  float x[4], y[4];
  a.get(x);
  b.get(y);
  return frag_of<NP>(f32x4{x[0], x[1], x[2], x[3]}, f32x4{y[0], y[1], y[2], y[3]});
}

template <typename T>
struct ChainArgs {
  Heads<const T> q, k, d_o;
  Heads<T> dv;
  const float *inverse, *gates, *ds1;
  float *ds, *ds0;  // every chunk's dS1, the initial state's gradient
};

template <typename T, int DK, int NW>
__global__ __launch_bounds__(64 * NW) void delta_chain_kernel(DeltaSizes z, ChainArgs<T> A, int n_blocks) {
  constexpr int kIn = DeltaType<T>::kIn, kLogC = DeltaType<T>::kLogC, C = 1 << kLogC;
  constexpr int RT = C / 16, KC = C / 32, DT = DK / 16, KD = DK / 32, kW = kStateWords;
  using RowImg = Image<RT, KD, kIn>;  // rows t, places d
  using ColImg = Image<DT, KC, kIn>;  // rows d, places t
  using SqImg = Image<RT, KC, kW>;    // rows j, places i: the inverse and P, transposed
  constexpr int kK = 0, kQ = kK + RowImg::kBytes, kKT = kQ + RowImg::kBytes, kQT = kKT + ColImg::kBytes,
                kInv = kQT + ColImg::kBytes, kP = kInv + SqImg::kBytes, kG = kP + SqImg::kBytes,
                kAll = kG + kGateRows * C * 4;
  __shared__ __align__(16) char lds[kAll];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, lg = lane >> 4;
  const int h = blockIdx.x / n_blocks, hk = h / (z.H / z.Hk), v0 = ((blockIdx.x % n_blocks) * NW + wave) * 16;
  const int s = blockIdx.y;
  const float* gate = reinterpret_cast<const float*>(lds + kG);
  uint32_t r0, r1, first;
  segment_rows(z.offs, s, static_cast<uint32_t>(z.T), kLogC, r0, r1, first);
  for (int i = threadIdx.x * 16; i < kG - kInv; i += 64 * NW * 16) *reinterpret_cast<u32x4*>(lds + kInv + i) = u32x4{0, 0, 0, 0};

  const int col = v0 + c;
  const bool live = col < z.dv;
  const int64_t size = static_cast<int64_t>(z.dk) * z.dv, of = (static_cast<int64_t>(s) * z.H + h) * size;
  f32x4 S[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = 16 * i + 4 * lg + r;
      S[i][r] = A.ds1 && live && d < z.dk ? A.ds1[of + static_cast<int64_t>(d) * z.dv + col] : 0.0f;
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

  constexpr int kThreads = 64 * NW, kRowBlocks = C * DK / 16, kInvBlocks = C * C / 16;
  constexpr int kNB = (kRowBlocks + kThreads - 1) / kThreads, kNI = (kInvBlocks + kThreads - 1) / kThreads;
  constexpr int kNG = (kGateRows * C + kThreads - 1) / kThreads;
  Raw4<T> rk[kNB][4], rq[kNB][4];
  f32x4 ri[kNI][4];
  float rg[kNG];
  T rd[RT][4];
  const auto fetch = [&](uint32_t t0, int64_t unit) {
    const int n = r1 - t0 < static_cast<uint32_t>(C) ? static_cast<int>(r1 - t0) : C;
#pragma unroll
    for (int b = 0; b < kNB; ++b) {
      const int id = b * kThreads + threadIdx.x, t = id / (DK / 4) * 4, d = id % (DK / 4) * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = id < kRowBlocks && t + j < n ? z.dk - d : 0;
        const int64_t row = m > 0 ? t0 + t + j : t0;
        rk[b][j].load(A.k.row(row, hk) + (m > 0 ? d : 0), m);
        rq[b][j].load(A.q.row(row, hk) + (m > 0 ? d : 0), m);
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
        rd[i][r] = live && t < n ? A.d_o.row(t0 + t, h)[col] : T{};
      }
  };

  const int chunks = static_cast<int>((r1 - r0 + C - 1) >> kLogC);
  const auto unit_of = [&](int i) { return (static_cast<int64_t>(first) + i) * z.H + h; };
  if (chunks) fetch(r0 + ((chunks - 1) << kLogC), unit_of(chunks - 1));
  for (int ch = chunks - 1; ch >= 0; --ch) {
    const uint32_t t0 = r0 + (static_cast<uint32_t>(ch) << kLogC);
    const int n = r1 - t0 < static_cast<uint32_t>(C) ? static_cast<int>(r1 - t0) : C;
    __syncthreads();  // the last chunk's fragments have been read
#pragma unroll
    for (int b = 0; b < kNB; ++b) {
      const int id = b * kThreads + threadIdx.x, t = id / (DK / 4) * 4, d = id % (DK / 4) * 4;
      if (id < kRowBlocks) {
        float x[4][4], y[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          rk[b][j].get(x[j]);
          RowImg::store4(lds + kK, t + j, d, x[j]);
          rq[b][j].get(y[j]);
          RowImg::store4(lds + kQ, t + j, d, y[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float w[4] = {x[0][j], x[1][j], x[2][j], x[3][j]}, u[4] = {y[0][j], y[1][j], y[2][j], y[3][j]};
          ColImg::store4(lds + kKT, d + j, t, w);
          ColImg::store4(lds + kQT, d + j, t, u);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kNI; ++b) {
      const int id = b * kThreads + threadIdx.x, i = id / (C / 4) * 4, j = id % (C / 4) * 4;
      if (id < kInvBlocks && j / 16 <= i / 16)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float w[4] = {ri[b][0][r], ri[b][1][r], ri[b][2][r], ri[b][3][r]};
          SqImg::store4(lds + kInv, j + r, i, w);
        }
    }
#pragma unroll
    for (int b = 0; b < kNG; ++b) {
      const int id = b * kThreads + threadIdx.x;
      if (id < kGateRows * C) reinterpret_cast<float*>(lds + kG)[id] = rg[b];
    }
    f32x4 dO[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) dO[i][r] = to_f32(rd[i][r]);
    __syncthreads();
    if (ch > 0) fetch(t0 - C, unit_of(ch - 1));
    write_state(A.ds + unit_of(ch) * size);

    // P transposed: rows i of the result are places of the image
    for (int p = wave; p < RT * (RT + 1) / 2; p += NW) {
      int i = 0, j = p;
      while (j > i) j -= ++i;
      f32x4 acc{};
#pragma unroll
      for (int ks = 0; ks < KD; ++ks)
        mm<kIn>(acc, RowImg::load(lds + kQ, i, ks), RowImg::load(lds + kK, j, ks));
      const int m = 16 * j + c;
      float w[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * lg + r;
        const float dcy = decay(gate[kGHi * C + row], gate[kGLo * C + row], gate[kGHi * C + m], gate[kGLo * C + m]);
        w[r] = m <= row ? acc[r] * dcy * z.scale : 0.0f;
      }
      SqImg::store4(lds + kP, m, 16 * i + 4 * lg, w);
    }
    f32x4 dU[RT] = {};
#pragma unroll
    for (int ks = 0; ks < KD; ++ks) {
      const Frag<kW> f = frag_of<kW>(S[2 * ks], S[2 * ks + 1]);
#pragma unroll
      for (int i = 0; i < RT; ++i) mm<kW>(dU[i], RowImg::load(lds + kK, i, ks), f);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) dU[i] *= gate4(gate, C, kRest, 16 * i + 4 * lg);
    __syncthreads();  // P is there
#pragma unroll
    for (int kt = 0; kt < KC; ++kt) {
      const Frag<kIn> f = frag_of<kIn>(dO[2 * kt], dO[2 * kt + 1]);
#pragma unroll
      for (int j = 0; j < RT && j < 2 * kt + 2; ++j) mm<kW>(dU[j], SqImg::load(lds + kP, j, kt), f);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) dU[i] *= gate4(gate, C, kBeta, 16 * i + 4 * lg);
    f32x4 dN[RT] = {};
#pragma unroll
    for (int kt = 0; kt < KC; ++kt) {
      const Frag<kW> f = frag_of<kW>(dU[2 * kt], dU[2 * kt + 1]);
#pragma unroll
      for (int j = 0; j < RT && j < 2 * kt + 2; ++j) mm<kW>(dN[j], SqImg::load(lds + kInv, j, kt), f);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * i + 4 * lg + r;
        if (live && t < n) A.dv.row(t0 + t, h)[col] = from_f32<T>(dN[i][r]);
      }
    const float el = gate[kEG * C + C - 1];
#pragma unroll
    for (int i = 0; i < DT; ++i) S[i] *= el;
#pragma unroll
    for (int kt = 0; kt < KC; ++kt) {
      const f32x4 e0 = gate4(gate, C, kEG, 32 * kt + 4 * lg), e1 = gate4(gate, C, kEG, 32 * kt + 16 + 4 * lg);
      const Frag<kW> fo = frag_of<kW>(dO[2 * kt] * (e0 * z.scale), dO[2 * kt + 1] * (e1 * z.scale));
      const Frag<kW> fn = frag_of<kW>(-dN[2 * kt] * e0, -dN[2 * kt + 1] * e1);
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        mm<kW>(S[i], ColImg::load(lds + kQT, i, kt), fo);
        mm<kW>(S[i], ColImg::load(lds + kKT, i, kt), fn);
      }
    }
  }
  if (A.ds0) write_state(A.ds0 + of);
}

template <typename T>
struct GradArgs {
  Heads<const T> q, k, v, d_o;
  Heads<T> dq, dk;
  T *dg, *dbeta;
  const float *g, *inverse, *gates, *states, *ds;
  int64_t g_ld, dg_ld, dbeta_ld;
};

// Workgroup (tile, hk): one chunk of one key head, its value heads in turn.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(4 * (DK > DV ? DK : DV)) void delta_grad_kernel(DeltaSizes z, GradArgs<T> A) {
  constexpr int kIn = DeltaType<T>::kIn, kW = DeltaType<T>::kOut, kLogC = DeltaType<T>::kLogC, C = 1 << kLogC;
  constexpr int NW = (DK > DV ? DK : DV) / 16, RT = C / 16, KC = C / 32, DT = DK / 16, KD = DK / 32, KV = DV / 32;
  constexpr int kPairs = RT * (RT + 1) / 2, kMine = (kPairs + NW - 1) / NW;  // tiles of token pairs, of a wave
  using KImg = Image<RT, KD, kIn>;  // rows t, places d
  using VImg = Image<RT, KV, kW>;   // rows t, places v
  using SqImg = Image<RT, KC, kW>;
  // the three square images hold P^T and the inverse both ways, then dP * D both ways and Z + Z^T
  constexpr int kK = 0, kN = kK + KImg::kBytes, kDN = kN + VImg::kBytes, kA = kDN + VImg::kBytes, kB = kA + SqImg::kBytes,
                kC = kB + SqImg::kBytes, kG = kC + SqImg::kBytes, kRed = kG + kGateRows * C * 4;
  constexpr int kPart = NW * C;  // one float per wave and row
  constexpr int kAll = kRed + (4 * kPart + 3 * kPairs * 16 + NW) * 4;
  __shared__ __align__(16) char lds[kAll];
  float* gate = reinterpret_cast<float*>(lds + kG);
  float *red_b = reinterpret_cast<float*>(lds + kRed), *red_n = red_b + kPart, *red_w = red_n + kPart, *red_q = red_w + kPart;
  float *row_e = red_q + kPart, *col_e = row_e + kPairs * 16, *col_x = col_e + kPairs * 16, *red_s = col_x + kPairs * 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, lg = lane >> 4;
  const uint32_t tile = blockIdx.x;
  const int hk = blockIdx.y, group = z.H / z.Hk;
  int e;
  uint32_t t0, t1, s0, s1;
  if (!segment_tile<1>(z.offs, z.S, static_cast<uint32_t>(z.T), kLogC, tile, e, t0, t1, s0, s1)) return;
  const int n = static_cast<int>(t1 - t0);
  const int64_t size = static_cast<int64_t>(z.dk) * z.dv;
  constexpr int kThreads = 64 * NW;

  // K as an image; the wave's channels of K and Q with tokens as places, in registers
  for (int id = threadIdx.x; id < C * DK / 4; id += kThreads) {
    const int t = id / (DK / 4), d = id % (DK / 4) * 4, m = t < n ? z.dk - d : 0;
    Raw4<T> w;
    w.load(A.k.row(t0 + (m > 0 ? t : 0), hk) + (m > 0 ? d : 0), m);
    float x[4];
    w.get(x);
    KImg::store4(lds + kK, t, d, x);
  }
  Frag<kIn> kT[KC], qT[KC];
  {
    const int d = 16 * wave + c;
#pragma unroll
    for (int kt = 0; kt < KC; ++kt) {
      f32x4 a[2], b[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 32 * kt + 16 * u + 4 * lg + r;
          const bool in = t < n && d < z.dk;
          a[u][r] = in ? to_f32(A.k.row(t0 + t, hk)[d]) : 0.0f;
          b[u][r] = in ? to_f32(A.q.row(t0 + t, hk)[d]) : 0.0f;
        }
      kT[kt] = frag_of<kIn>(a[0], a[1]);
      qT[kt] = frag_of<kIn>(b[0], b[1]);
    }
  }
  f32x4 dq[RT] = {}, dk[RT] = {};  // rows d, columns t

  for (int h = hk * group; h < (hk + 1) * group; ++h) {
    const int64_t unit = static_cast<int64_t>(tile) * z.H + h;
    __syncthreads();  // the last head's images and sums have been read
    {
      const float* inv = A.inverse + unit * (C * C);
      for (int id = threadIdx.x; id < C * C / 16; id += kThreads) {
        const int i = id / (C / 4) * 4, j = id % (C / 4) * 4;
        const bool in = j / 16 <= i / 16;
        f32x4 x[4] = {};
        if (in)
#pragma unroll
          for (int r = 0; r < 4; ++r) x[r] = *reinterpret_cast<const f32x4*>(inv + (i + r) * C + j);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float w[4] = {x[r][0], x[r][1], x[r][2], x[r][3]}, u[4] = {x[0][r], x[1][r], x[2][r], x[3][r]};
          SqImg::store4(lds + kB, i + r, j, w);
          SqImg::store4(lds + kC, j + r, i, u);
        }
      }
      for (int id = threadIdx.x; id < kGateRows * C; id += kThreads) gate[id] = A.gates[unit * (kGateRows * C) + id];
    }
    __syncthreads();

    // The wave's tiles of token pairs: rows j, columns i.
    f32x4 P[kMine], M[kMine], D[kMine];
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int p = wave + m * NW;
      if (p < kPairs) {
        int i = 0, j = p;
        while (j > i) j -= ++i;
        f32x4 qk{}, kk{};
        const int row = 16 * i + c;
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) {
          const Frag<kIn> kj = KImg::load(lds + kK, j, ks);
          mm<kIn>(kk, kj, KImg::load(lds + kK, i, ks));
          mm<kIn>(qk, kj, row_frag<kIn>(A.q.row(t0 + (row < n ? row : 0), hk), row < n ? z.dk : 0, ks));
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = 16 * j + 4 * lg + r;
          const float dcy = decay(gate[kGHi * C + row], gate[kGLo * C + row], gate[kGHi * C + at], gate[kGLo * C + at]);
          D[m][r] = at <= row ? dcy : 0.0f;
          P[m][r] = at <= row ? qk[r] * dcy * z.scale : 0.0f;
          M[m][r] = at < row ? kk[r] * dcy : 0.0f;
          SqImg::store1(lds + kA, at, row, P[m][r]);  // rows j, places i
          if (i != j) SqImg::store1(lds + kA, row, at, 0.0f);
        }
      }
    }
    __syncthreads();

    // 16 columns of v: N, dU, dN
    if (wave < DV / 16) {
      const int col = 16 * wave + c;
      const bool live = col < z.dv;
      f32x4 N[RT], dN[RT] = {}, dU[RT] = {};
      float inner = 0.0f;
      {
        f32x4 R[RT], dO[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int t = 16 * i + 4 * lg + r;
            const bool in = live && t < n;
            R[i][r] = in ? to_f32(A.v.row(t0 + t, h)[col]) : 0.0f;
            dO[i][r] = in ? to_f32(A.d_o.row(t0 + t, h)[col]) : 0.0f;
          }
        f32x4 ks0[RT] = {};
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) {
          f32x4 a[2], b[2];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int d = 32 * ks + 16 * u + 4 * lg + r;
              const bool in = live && d < z.dk;
              const int64_t at = unit * size + static_cast<int64_t>(d) * z.dv + col;
              a[u][r] = in ? A.states[at] : 0.0f;
              b[u][r] = in ? A.ds[at] : 0.0f;
              inner = __builtin_fmaf(a[u][r], b[u][r], inner);
            }
          const Frag<kW> fs = frag_of<kW>(a[0], a[1]), fd = frag_of<kW>(b[0], b[1]);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const Frag<kIn> f = KImg::load(lds + kK, i, ks);
            mm<kW>(ks0[i], f, fs);
            mm<kW>(dU[i], f, fd);
          }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          ks0[i] *= gate4(gate, C, kEG, 16 * i + 4 * lg);
          dU[i] *= gate4(gate, C, kRest, 16 * i + 4 * lg);
          R[i] -= ks0[i];
          N[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int kt = 0; kt < KC; ++kt) {
          const Frag<kW> f = frag_of<kW>(R[2 * kt], R[2 * kt + 1]);
#pragma unroll
          for (int i = 2 * kt; i < RT; ++i) mm<kW>(N[i], SqImg::load(lds + kB, i, kt), f);
        }
        // w, before P^T dO joins dU
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const f32x4 b = gate4(gate, C, kBeta, 16 * i + 4 * lg);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float w = row16_tree(b[r] * N[i][r] * dU[i][r]);
            if (c == 0) red_w[wave * C + 16 * i + 4 * lg + r] = w;
          }
        }
#pragma unroll
        for (int kt = 0; kt < KC; ++kt) {
          const Frag<kIn> f = frag_of<kIn>(dO[2 * kt], dO[2 * kt + 1]);
#pragma unroll
          for (int j = 0; j < RT && j < 2 * kt + 2; ++j) mm<kW>(dU[j], SqImg::load(lds + kA, j, kt), f);
        }
#pragma unroll
        for (int kt = 0; kt < KC; ++kt) {
          const f32x4 b0 = gate4(gate, C, kBeta, 32 * kt + 4 * lg), b1 = gate4(gate, C, kBeta, 32 * kt + 16 + 4 * lg);
          const Frag<kW> f = frag_of<kW>(dU[2 * kt] * b0, dU[2 * kt + 1] * b1);
#pragma unroll
          for (int j = 0; j < RT && j < 2 * kt + 2; ++j) mm<kW>(dN[j], SqImg::load(lds + kC, j, kt), f);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float b = row16_tree(dU[i][r] * N[i][r]), m = row16_tree(dN[i][r] * ks0[i][r]);
            const int t = 16 * i + 4 * lg + r;
            if (c == 0) {
              red_b[wave * C + t] = b;
              red_n[wave * C + t] = m;
            }
            VImg::store1(lds + kN, t, col, N[i][r]);
            VImg::store1(lds + kDN, t, col, dN[i][r]);
          }
      }
      inner = lanes_sum<64>(inner);
      if (lane == 0) red_s[wave] = inner;
    }
    __syncthreads();

    // The pair tiles: dP, X and what comes of them.
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int p = wave + m * NW;
      if (p < kPairs) {
        int i = 0, j = p;
        while (j > i) j -= ++i;
        f32x4 x{}, y{};
        const int row = 16 * i + c;
#pragma unroll
        for (int kv = 0; kv < KV; ++kv) {
          const Frag<kW> f = VImg::load(lds + kN, j, kv);
          mm<kW>(x, f, VImg::load(lds + kDN, i, kv));
          mm<kW>(y, f, row_frag<kIn>(A.d_o.row(t0 + (row < n ? row : 0), h), row < n ? z.dv : 0, kv));
        }
        const f32x4 b = gate4(gate, C, kBeta, 16 * j + 4 * lg);
        f32x4 pd, zz, ev, mx;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = 16 * j + 4 * lg + r;
          pd[r] = at <= row ? b[r] * y[r] * D[m][r] * z.scale : 0.0f;
          zz[r] = at < row ? -b[r] * x[r] * D[m][r] : 0.0f;
          mx[r] = at < row ? M[m][r] * x[r] : 0.0f;
          ev[r] = (at <= row ? b[r] * y[r] * P[m][r] : 0.0f) - b[r] * mx[r];
        }
        // sums over j (rows of the tile) for row i, over i (its columns) for row j
        float s = (ev[0] + ev[1]) + (ev[2] + ev[3]);
        const Halves s16 = halves16(s);
        const Halves s32 = halves32(s16.a + s16.b);
        if (lg == 0) row_e[p * 16 + c] = s32.a + s32.b;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float ce = row16_tree(ev[r]), cx = row16_tree(mx[r]);
          if (c == 0) {
            col_e[p * 16 + 4 * lg + r] = ce;
            col_x[p * 16 + 4 * lg + r] = cx;
          }
        }
        const float w[4] = {pd[0], pd[1], pd[2], pd[3]};
        SqImg::store4(lds + kA, row, 16 * j + 4 * lg, w);  // dP * D: rows i, places j
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = 16 * j + 4 * lg + r;
          SqImg::store1(lds + kB, at, row, pd[r]);  // rows j, places i
          if (i != j || at <= row) {
            SqImg::store1(lds + kC, row, at, zz[r]);
            SqImg::store1(lds + kC, at, row, zz[r]);
          }
          if (i != j) {  // the tiles on the far side of the diagonal
            SqImg::store1(lds + kA, at, row, 0.0f);
            SqImg::store1(lds + kB, row, at, 0.0f);
          }
        }
      }
    }
    __syncthreads();

    // 16 channels of dq and dk
    if (wave < DT) {
      f32x4 a[RT] = {}, b[RT] = {}, s[RT] = {};
      const int d = 16 * wave + c;
      const float* ps = A.states + unit * size + static_cast<int64_t>(d < z.dk ? d : 0) * z.dv;
      const float* pd = A.ds + unit * size + static_cast<int64_t>(d < z.dk ? d : 0) * z.dv;
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) {
        const Frag<kW> fs = row_frag<kW>(ps, d < z.dk ? z.dv : 0, kv), fd = row_frag<kW>(pd, d < z.dk ? z.dv : 0, kv);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const int t = 16 * i + c;
          mm<kW>(a[i], fs, row_frag<kIn>(A.d_o.row(t0 + (t < n ? t : 0), h), t < n ? z.dv : 0, kv));
          mm<kW>(b[i], fs, VImg::load(lds + kDN, i, kv));
          mm<kW>(s[i], fd, VImg::load(lds + kN, i, kv));
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int t = 16 * i + c;
        const float eg = gate[kEG * C + t], w = gate[kRest * C + t] * gate[kBeta * C + t];
        a[i] *= eg * z.scale;
        // this wave's part of dO . (scale e^G Q S0) = q . (its part of dq)
        Raw4<T> rq;
        const int m = t < n ? z.dk - 16 * wave - 4 * lg : 0;
        rq.load(A.q.row(t0 + (m > 0 ? t : 0), hk) + (m > 0 ? 16 * wave + 4 * lg : 0), m);
        float q[4];
        rq.get(q);
        float dot = (q[0] * a[i][0] + q[1] * a[i][1]) + (q[2] * a[i][2] + q[3] * a[i][3]);
        const Halves h16 = halves16(dot);
        const Halves h32 = halves32(h16.a + h16.b);
        if (lg == 0) red_q[wave * C + t] = h32.a + h32.b;
        dk[i] += s[i] * w - b[i] * eg;
        dq[i] += a[i];
      }
#pragma unroll
      for (int kt = 0; kt < KC; ++kt)
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          if (i >= 2 * kt) mm<kW>(dq[i], kT[kt], SqImg::load(lds + kA, i, kt));
          if (i < 2 * kt + 2) mm<kW>(dk[i], qT[kt], SqImg::load(lds + kB, i, kt));
          mm<kW>(dk[i], kT[kt], SqImg::load(lds + kC, i, kt));
        }
    }
    __syncthreads();

    // dbeta and dg, by the first wave: a lane per token
    if (wave == 0) {
      const int t = lane < C ? lane : 0, rt = t / 16, q = t % 16;
      float db = 0.0f, w = 0.0f, dG = 0.0f, inner = 0.0f;
#pragma unroll
      for (int i = 0; i < DV / 16; ++i) {
        db += red_b[i * C + t];
        w += red_w[i * C + t];
        dG -= red_n[i * C + t];
        inner += red_s[i];
      }
#pragma unroll
      for (int i = 0; i < DT; ++i) dG += red_q[i * C + t];
      dG -= w;
      for (int j = 0; j <= rt; ++j) dG += row_e[(rt * (rt + 1) / 2 + j) * 16 + q];
      for (int i = rt; i < RT; ++i) {
        dG -= col_e[(i * (i + 1) / 2 + rt) * 16 + q];
        db -= col_x[(i * (i + 1) / 2 + rt) * 16 + q];
      }
      // the sums from a row to the end, in float64
      double sum = lane < C ? static_cast<double>(dG) : 0.0, all = lane < C ? static_cast<double>(w) : 0.0;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) all += __shfl_xor(all, d);
      if (lane == C - 1) sum += all + static_cast<double>(gate[kEG * C + C - 1]) * inner;
#pragma unroll
      for (int d = 1; d < C; d <<= 1) {
        const double o = __shfl_down(sum, d);
        if (lane + d < C) sum += o;
      }
      if (lane < n) {
        const bool cut = A.g[(t0 + t) * A.g_ld + h] < -104.0f;
        A.dg[(t0 + t) * A.dg_ld + h] = from_f32<T>(cut ? 0.0f : static_cast<float>(sum));
        A.dbeta[(t0 + t) * A.dbeta_ld + h] = from_f32<T>(db);
      }
    }
  }
  if (wave < DT) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int t = 16 * i + c, d = 16 * wave + 4 * lg;
      if (t < n && d < z.dk) {
        store4(A.dq.row(t0 + t, hk) + d, z.dk - d, dq[i]);
        store4(A.dk.row(t0 + t, hk) + d, z.dk - d, dk[i]);
      }
    }
  }
}

struct Layout {
  size_t inverse, gates, ds, all;
};
Layout layout_of(const DeltaSizes& z, int dtype) {
  const int64_t C = dtype == DET_BF16 ? 64 : 32, units = delta_tiles(z.T, z.S, dtype) * z.H;
  Layout l;
  l.inverse = DET_WS_HEADER_BYTES;
  l.gates = l.inverse + static_cast<size_t>(units * C * C) * 4;
  l.ds = l.gates + align_up(static_cast<size_t>(units * kGateRows * C) * 4, 256);
  l.all = l.ds + align_up(static_cast<size_t>(units * z.dk * z.dv) * 4, 256);
  return l;
}

template <typename T, int DK>
void launch_chain(const DeltaSizes& z, const ChainArgs<T>& A, hipStream_t st) {
  int nw = 8;
  while (nw > 1 && (static_cast<int64_t>(z.S) * z.H * ceil_div(z.dv, 16 * nw) < 256 || 16 * nw >= 2 * z.dv)) nw /= 2;
  const int n_blocks = static_cast<int>(ceil_div(z.dv, 16 * nw));
  const dim3 grid(static_cast<uint32_t>(z.H * n_blocks), static_cast<uint32_t>(z.S));
#define DET_DELTA_CHAIN(NW) \
  case NW: hipLaunchKernelGGL((delta_chain_kernel<T, DK, NW>), grid, dim3(64 * NW), 0, st, z, A, n_blocks); break;
  switch (nw) {
    DET_DELTA_CHAIN(1)
    DET_DELTA_CHAIN(2)
    DET_DELTA_CHAIN(4)
    DET_DELTA_CHAIN(8)
  }
#undef DET_DELTA_CHAIN
}

template <typename T, int DK, int DV>
void launch_grad(const DeltaSizes& z, const GradArgs<T>& A, int dtype, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(delta_tiles(z.T, z.S, dtype)), static_cast<uint32_t>(z.Hk));
  hipLaunchKernelGGL((delta_grad_kernel<T, DK, DV>), grid, dim3(4 * (DK > DV ? DK : DV)), 0, st, z, A);
}

}  // namespace
}  // namespace detgrad

using namespace detgrad;

extern "C" int det_delta_rule_bwd_workspace_size(int64_t T, int64_t S, int64_t H, int64_t dk, int64_t dv, int dtype,
                                                 size_t* bytes) {
  if (!bytes) return set_error(DET_ERR_INVALID_ARG, "delta_rule_bwd: bytes is NULL");
  if (int s = delta_check_sizes("delta_rule_bwd", dtype, T, S, 1, H, dk, dv)) return s;
  const DeltaSizes z{T, (int)S, 1, (int)H, (int)dk, (int)dv, nullptr, 0.0f};
  *bytes = T == 0 ? 0 : layout_of(z, dtype).all;
  return ok();
}

extern "C" int det_delta_rule_bwd(const void* d_o, int64_t do_st, int64_t do_sh, const void* q, int64_t q_st, int64_t q_sh,
                                  const void* k, int64_t k_st, int64_t k_sh, const void* v, int64_t v_st, int64_t v_sh,
                                  const float* g, int64_t g_ld, const void* beta, int64_t beta_ld, int dtype, int64_t T,
                                  int64_t Hk, int64_t H, int64_t dk, int64_t dv, const int32_t* offs, int64_t S, double scale,
                                  const float* states, const float* dfinal_state, void* dq, int64_t dq_st, int64_t dq_sh,
                                  void* dk_out, int64_t dk_st, int64_t dk_sh, void* dv_out, int64_t dv_st, int64_t dv_sh,
                                  void* dg, int64_t dg_ld, void* dbeta, int64_t dbeta_ld, float* dinitial_state, void* ws,
                                  size_t ws_bytes, void* stream) {
  const char* what = "delta_rule_bwd";
  if (int s = delta_check_sizes(what, dtype, T, S, Hk, H, dk, dv)) return s;
  if (!(scale > -1e30 && scale < 1e30)) return set_error(DET_ERR_INVALID_ARG, "%s: scale must be finite", what);
  if (S == 0) return ok();
  if (!offs || (T > 0 && (!d_o || !q || !k || !v || !g || !beta || !states || !dq || !dk_out || !dv_out || !dg || !dbeta)))
    return set_error(DET_ERR_INVALID_ARG, "%s: NULL pointer", what);
  const size_t es = dtype_size(dtype);
  Buf b[7];
  if (int s = delta_buf(what, "do", d_o, T, H, dv, do_st, do_sh, es, b[0])) return s;
  if (int s = delta_buf(what, "q", q, T, Hk, dk, q_st, q_sh, es, b[1])) return s;
  if (int s = delta_buf(what, "k", k, T, Hk, dk, k_st, k_sh, es, b[2])) return s;
  if (int s = delta_buf(what, "v", v, T, H, dv, v_st, v_sh, es, b[3])) return s;
  if (int s = delta_buf(what, "dq", dq, T, Hk, dk, dq_st, dq_sh, es, b[4])) return s;
  if (int s = delta_buf(what, "dk", dk_out, T, Hk, dk, dk_st, dk_sh, es, b[5])) return s;
  if (int s = delta_buf(what, "dv", dv_out, T, H, dv, dv_st, dv_sh, es, b[6])) return s;
  const int64_t lds_[] = {g_ld, beta_ld, dg_ld, dbeta_ld};
  for (int64_t ld : lds_) {
    if (T > 1 && ld < H) return set_error(DET_ERR_INVALID_ARG, "%s: row stride of g, beta, dg or dbeta < H", what);
    if (T > 0 && ld > (int64_t(1) << 44) / T) return set_error(DET_ERR_UNSUPPORTED, "%s: g, beta, dg or dbeta is too large", what);
  }
  const DeltaSizes z{T, (int)S, (int)Hk, (int)H, (int)dk, (int)dv, offs, static_cast<float>(scale)};
  const Layout l = layout_of(z, dtype);
  const size_t need = T ? l.all : 0;
  if (int s = check_workspace(ws, ws_bytes, need)) return s;
  const size_t state = static_cast<size_t>(H * dk * dv) * 4;
  const auto gates = [&](const char* name, const void* p, int64_t ld, size_t el) {
    return buf_rows(name, p, T, H, T > 1 ? ld : H, el);
  };
  const Buf outs[] = {b[4], b[5], b[6], gates("dg", dg, dg_ld, es), gates("dbeta", dbeta, dbeta_ld, es),
                      {"dinitial_state", range1d(dinitial_state, S * state)},
                      {"the workspace", range1d(need ? ws : nullptr, ws_bytes)}};
  const Buf ins[] = {b[0], b[1], b[2], b[3], gates("g", g, g_ld, 4), gates("beta", beta, beta_ld, es),
                     {"offs", range1d(offs, (S + 1) * 4)},
                     {"states", range1d(states, delta_tiles(T, S, dtype) * state)},
                     {"dfinal_state", range1d(dfinal_state, S * state)}};
  if (int s = check_buffers(what, outs, 7, ins, 9)) return s;
  const hipStream_t st = as_stream(stream);
  float *inverse = nullptr, *gate = nullptr, *ds = nullptr;
  if (T) {
    char* p = static_cast<char*>(ws);
    inverse = reinterpret_cast<float*>(p + l.inverse);
    gate = reinterpret_cast<float*>(p + l.gates);
    ds = reinterpret_cast<float*>(p + l.ds);
    delta_prepare(z, dtype, k, k_st, k_sh, g, g_ld, beta, beta_ld, inverse, gate, st);
  }
#define DET_DELTA_BWD(E)                                                                                               \
  {                                                                                                                    \
    const Heads<const E> hq{static_cast<const E*>(q), q_st, q_sh}, hk{static_cast<const E*>(k), k_st, k_sh},           \
        hv{static_cast<const E*>(v), v_st, v_sh}, ho{static_cast<const E*>(d_o), do_st, do_sh};                        \
    const ChainArgs<E> A{hq, hk, ho, {static_cast<E*>(dv_out), dv_st, dv_sh}, inverse, gate, dfinal_state, ds,         \
                         dinitial_state};                                                                              \
    const GradArgs<E> B{hq, hk, hv, ho, {static_cast<E*>(dq), dq_st, dq_sh}, {static_cast<E*>(dk_out), dk_st, dk_sh},  \
                        static_cast<E*>(dg), static_cast<E*>(dbeta), g, inverse, gate, states, ds, g_ld, dg_ld,        \
                        dbeta_ld};                                                                                     \
    if (dk <= 64) launch_chain<E, 64>(z, A, st);                                                                       \
    else launch_chain<E, 128>(z, A, st);                                                                               \
    if (T) {                                                                                                           \
      if (dk <= 64 && dv <= 64) launch_grad<E, 64, 64>(z, B, dtype, st);                                               \
      else if (dk <= 64) launch_grad<E, 64, 128>(z, B, dtype, st);                                                     \
      else if (dv <= 64) launch_grad<E, 128, 64>(z, B, dtype, st);                                                     \
      else launch_grad<E, 128, 128>(z, B, dtype, st);                                                                  \
    }                                                                                                                  \
  }
  if (dtype == DET_BF16) DET_DELTA_BWD(uint16_t)
  else DET_DELTA_BWD(float)
#undef DET_DELTA_BWD
  return check_launch("det_delta_rule_bwd");
}
