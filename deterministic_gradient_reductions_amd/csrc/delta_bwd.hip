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
// Nothing is divided by beta or by a decay. After the forward's two preparing kernels
// (with P and the inverse transposed too) one kernel walks a sequence's chunks backwards
// as the forward's walks them (16 columns of v per wave, dS in registers) and writes
// every chunk's dS1, and one takes all chunks side by side: it forms N, dU and dN of its
// chunk again and the sums over v and over token pairs. There a wave owns 16 columns of
// v first (N, dN), then tiles of token pairs, then 16 channels of dQ and dK; N, dN and
// the pair matrices change hands in LDS as images.
#include "delta.hpp"

namespace detgrad {
namespace {

__device__ __forceinline__ f32x4 gate4(const float* gate, int C, int row, int at) {
  return *reinterpret_cast<const f32x4*>(gate + row * C + at);
}

template <typename T>
struct ChainArgs {
  Rows k;
  Heads<const T> d_o;
  const uint16_t *k_t, *q_t, *inverse_t, *p_t;
  const float *gates, *ds1;
  float *ds, *ds0;  // every chunk's dS1, the initial state's gradient
};

// Workgroups, waves and buffers as in the forward's chain; K^T and Q^T have one buffer.
template <typename T, int DK, int NW>
__global__ __launch_bounds__(64 * NW) void delta_chain_kernel(DeltaSizes z, ChainArgs<T> A) {
  constexpr int kIn = DeltaType<T>::kIn, kLogC = DeltaType<T>::kLogC, C = 1 << kLogC;
  constexpr int RT = C / 16, KC = C / 32, DT = DK / 16, KD = DK / 32, kW = kStateWords, kFrags = KC * (KC + 1);
  constexpr int nRows = RT * KD * kIn, nSq = kFrags * kW, nGate = (kGateRows * C * 4 + 1023) / 1024, nT = DT * KC * kIn;
  constexpr int oInv = nRows, oP = oInv + nSq, oGate = oP + nSq, kBuf = (oGate + nGate) * 1024;
  __shared__ __align__(16) char lds[2 * kBuf + 2 * nT * 1024];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, lg = lane >> 4;
  const int h = blockIdx.x % z.H, hk = h / (z.H / z.Hk), v0 = ((blockIdx.x / z.H) * NW + wave) * 16, s = blockIdx.y;
  const uint32_t lds0 = lds_address(lds);
  const char *kt_img = lds + 2 * kBuf, *qt_img = kt_img + nT * 1024;
  uint32_t r0, r1, first;
  segment_rows(z.offs, s, static_cast<uint32_t>(z.T), kLogC, r0, r1, first);
  const int col = v0 + c, vcol = col < z.dv ? col : z.dv - 1;
  const int64_t size = static_cast<int64_t>(z.dk) * z.dv, of = (static_cast<int64_t>(s) * z.H + h) * size;
  f32x4 S[DT] = {};
  if (A.ds1) {
    float x[DT][4];
    load_state<DT>(x, A.ds1 + of, z.dk, z.dv, vcol);
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = rho(i, 4 * lg + r) < z.dk ? x[i][r] : 0.0f;
  }
  T rd[RT][4];
  const auto fetch = [&](uint32_t t0, int64_t unit, int buf) {
    const int last = (r1 - t0 < static_cast<uint32_t>(C) ? static_cast<int>(r1 - t0) : C) - 1;
    load_column<RT>(rd, A.d_o.row(t0, h), A.d_o.st, vcol, last);
    const uint32_t to = lds0 + buf * kBuf;
    fetch_rows<RT, KD, kIn, NW>(to, A.k, t0, last, hk, wave);
    fetch_image<nSq, NW>(to + oInv * 1024, A.inverse_t + unit * (nSq * kFragElems), wave);
    fetch_image<nSq, NW>(to + oP * 1024, A.p_t + unit * (nSq * kFragElems), wave);
    fetch_image<nGate, NW>(to + oGate * 1024, reinterpret_cast<const uint16_t*>(A.gates + unit * (kGateRows * C)), wave);
  };
  const int chunks = static_cast<int>((r1 - r0 + C - 1) >> kLogC);
  const auto start = [&](int ch) { return r0 + (static_cast<uint32_t>(ch) << kLogC); };
  int64_t unit = (static_cast<int64_t>(first) + chunks - 1) * z.H + h;
  int buf = 0;
  if (chunks) fetch(start(chunks - 1), unit, 0);
  fetch_done();
  for (int ch = chunks - 1; ch >= 0; --ch, unit -= z.H, buf ^= 1) {
    f32x4 dU[RT] = {}, dO[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) dO[i][r] = to_f32(rd[i][r]);
    __syncthreads();  // this chunk's fragments are there, the last one's have been read
    const int64_t at = (unit / z.H * z.Hk + hk) * (nT * kFragElems);
    fetch_image<nT, NW>(lds0 + 2 * kBuf, A.k_t + at, wave);
    fetch_image<nT, NW>(lds0 + 2 * kBuf + nT * 1024, A.q_t + at, wave);
    if (ch > 0) fetch(start(ch - 1), unit - z.H, buf ^ 1);
    store_state<DT>(S, A.ds + unit * size, z.dk, z.dv, col);
    const char* img = lds + buf * kBuf;
    const float* gate = reinterpret_cast<const float*>(img + oGate * 1024);
#pragma unroll
    for (int ks = 0; ks < KD; ++ks) {
      const Frag<kW> f = frag_of<kW>(S[2 * ks], S[2 * ks + 1]);
      Frag<kIn> fk[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) fk[i] = lds_frag<kIn, kIn>(img, i * KD + ks);
      mm_tiles<kW, 0, RT>(dU, fk, f);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) dU[i] *= gate4(gate, C, kRest, rho(i, 4 * lg));
    static_for<KC>([&](auto kt) {
      constexpr int to = 2 * kt.value + 2;
      const Frag<kIn> f = frag_of<kIn>(dO[2 * kt.value], dO[2 * kt.value + 1]);
      Frag<kW> fp[RT];
#pragma unroll
      for (int j = 0; j < to; ++j) fp[j] = lds_frag<kW, kW>(img + oP * 1024, upper_frag<KC>(j, kt.value));
      mm_tiles<kW, 0, to>(dU, fp, f);
    });
    f32x4 dN[RT] = {};
#pragma unroll
    for (int i = 0; i < RT; ++i) dU[i] *= gate4(gate, C, kBeta, rho(i, 4 * lg));
    static_for<KC>([&](auto kt) {
      constexpr int to = 2 * kt.value + 2;
      const Frag<kW> f = frag_of<kW>(dU[2 * kt.value], dU[2 * kt.value + 1]);
      Frag<kW> fi[RT];
#pragma unroll
      for (int j = 0; j < to; ++j) fi[j] = lds_frag<kW, kW>(img + oInv * 1024, upper_frag<KC>(j, kt.value));
      mm_tiles<kW, 0, to>(dN, fi, f);
    });
    const float el = gate[kEnd * C];
#pragma unroll
    for (int i = 0; i < DT; ++i) S[i] *= el;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const f32x4 eg = gate4(gate, C, kEG, rho(i, 4 * lg));
      dO[i] *= eg * z.scale;
      dN[i] *= -eg;
    }
    fetch_done();
    __syncthreads();  // K^T and Q^T are there, and the next chunk's fragments
#pragma unroll
    for (int kt = 0; kt < KC; ++kt) {
      const Frag<kW> fo = frag_of<kW>(dO[2 * kt], dO[2 * kt + 1]), fn = frag_of<kW>(dN[2 * kt], dN[2 * kt + 1]);
      Frag<kIn> fq[DT], fk[DT];
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        fq[i] = lds_frag<kIn, kIn>(qt_img, i * KC + kt);
        fk[i] = lds_frag<kIn, kIn>(kt_img, i * KC + kt);
      }
      mm_tiles<kW, 0, DT>(S, fq, fo);
      mm_tiles<kW, 0, DT>(S, fk, fn);
    }
  }
  if (A.ds0) store_state<DT>(S, A.ds0 + of, z.dk, z.dv, col);
}

template <typename T>
struct GradArgs {
  Rows k, q, d_o_rows;
  Heads<const T> v, d_o;
  Heads<T> dq, dk, dv;
  T *dg, *dbeta;
  const uint16_t *k_t, *q_t, *inverse, *inverse_t, *p_t;
  const float *g, *gates, *states, *ds;
  int64_t g_ld, dg_ld, dbeta_ld;
};

// No instruction is moved over this: what a step loads is not loaded steps before, in
// registers that the steps between need.
__device__ __forceinline__ void step() { __builtin_amdgcn_sched_barrier(0); }

// Pair tile p: tiles i of rows and j of columns of the lower triangle, whole blocks of 32.
__device__ __forceinline__ void pair_of(int p, int& i, int& j) {
  i = p < 4 ? p >> 1 : 2 + ((p - 4) >> 2);
  j = p < 4 ? p & 1 : (p - 4) & 3;
}

// Workgroup (tile, hk): one chunk of one key head, its value heads in turn. What the
// products over channels and the chunk's squares need comes to LDS, the rest of a
// phase's operands to registers all at once, a phase ahead where there is room: the
// kernel's time goes into memory's latency otherwise (3583 us against ... at 16384
// tokens of 32 heads, 128 x 128).
template <typename T, int DK, int DV>
__global__ __launch_bounds__(4 * (DK > DV ? DK : DV), DK > DV ? DK / 64 : DV / 64) void delta_grad_kernel(DeltaSizes z,
                                                                                                       GradArgs<T> A) {
  constexpr int kIn = DeltaType<T>::kIn, kW = DeltaType<T>::kOut, kSW = kStateWords, kLogC = DeltaType<T>::kLogC, C = 1 << kLogC;
  constexpr int NW = (DK > DV ? DK : DV) / 16, RT = C / 16, KC = C / 32, DT = DK / 16, KD = DK / 32, KV = DV / 32;
  constexpr int kFrags = KC * (KC + 1), kPairs = 2 * kFrags, kMine = (kPairs + NW - 1) / NW;  // pair tiles, of a wave
  // 1024-byte fragments of the images
  constexpr int nRows = RT * KD * kIn, nV = RT * KV * kW, nSq = RT * KC * kW, nTri = kFrags * kSW, nGate = (kGateRows * C * 4 + 1023) / 1024;
  // the pair matrices take the place of the inverses and of P
  constexpr int nShared = 3 * nSq > 3 * nTri ? 3 * nSq : 3 * nTri;
  constexpr int oN = nRows, oDN = oN + nV, oS = oDN + nV, oGate = oS + nShared, nAll = oGate + nGate;
  __shared__ __align__(16) char lds[nAll * 1024];
  __shared__ float red_b[NW][C], red_n[NW][C], red_q[NW][C], red_s[NW], red_w[NW];
  __shared__ float row_e[RT][RT][16], col_e[RT][RT][16], col_x[RT][RT][16];
  const float* gate = reinterpret_cast<const float*>(lds + oGate * 1024);
  char *img_a = lds + oS * 1024, *img_b = img_a + nSq * 1024, *img_c = img_b + nSq * 1024;
  const char *inv = img_a, *inv_t = img_a + nTri * 1024, *p_t = inv_t + nTri * 1024;
  const uint32_t lds0 = lds_address(lds);
  const int wave_ = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = blockIdx.x;
  const int hk = blockIdx.y, group = z.H / z.Hk;
  int e;
  uint32_t t0, t1, s0, s1;
  if (!segment_tile<1>(z.offs, z.S, static_cast<uint32_t>(z.T), kLogC, tile, e, t0, t1, s0, s1)) return;
  const int size = z.dk * z.dv;
  const bool full = z.dk == DK && z.dv == DV;  // no padded channel
  constexpr int kThreads = 64 * NW;
  fetch_rows<RT, KD, kIn, NW>(lds0, A.k, t0, static_cast<int>(t1 - t0) - 1, hk, wave_);
  f32x4 dq[RT] = {}, dk[RT] = {};  // rows d, columns t

  for (int h = hk * group; h < (hk + 1) * group; ++h) {
    const int wave = here(wave_), lane = here_lane(threadIdx.x) & 63, c = lane & 15, lg = lane >> 4;
    const int n = here(static_cast<int>(t1 - t0));
    const int64_t unit = static_cast<int64_t>(tile) * z.H + h;
    const float *ps = A.states + unit * size, *pd = A.ds + unit * size;
    __syncthreads();  // the last head's images and sums have been read
    fetch_image<nTri, NW>(lds0 + oS * 1024, A.inverse + unit * (nTri * kFragElems), wave);
    fetch_image<nTri, NW>(lds0 + (oS + nTri) * 1024, A.inverse_t + unit * (nTri * kFragElems), wave);
    fetch_image<nTri, NW>(lds0 + (oS + 2 * nTri) * 1024, A.p_t + unit * (nTri * kFragElems), wave);
    fetch_image<nGate, NW>(lds0 + oGate * 1024, reinterpret_cast<const uint16_t*>(A.gates + unit * (kGateRows * C)), wave);

    // 16 columns of v: N, dU, dN
    const int col = 16 * wave + c, vcol = col < z.dv ? col : z.dv - 1;
    const bool live = col < z.dv;
    T rv[RT][4], ro[RT][4];
    float rs[DT][4], rd[DT][4];
    if (wave < DV / 16) {
      load_column<RT>(rv, A.v.row(t0, h), A.v.st, vcol, n - 1);
      load_column<RT>(ro, A.d_o.row(t0, h), A.d_o.st, vcol, n - 1);
      load_state<DT>(rs, ps, z.dk, z.dv, vcol);
      load_state<DT>(rd, pd, z.dk, z.dv, vcol);
    }
    fetch_done();
    __syncthreads();
    if (wave < DV / 16) {
      f32x4 N[RT] = {}, dN[RT] = {}, dU[RT] = {}, ks0[RT] = {}, dO[RT];
      float inner = 0.0f, w_sum = 0.0f;
      if (!full)
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool in = live && rho(i, 4 * lg + r) < z.dk;
            rs[i][r] = in ? rs[i][r] : 0.0f;
            rd[i][r] = in ? rd[i][r] : 0.0f;
          }
#pragma unroll
      for (int ks = 0; ks < KD; ++ks) {
        f32x4 a[2], b[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            a[u][r] = rs[2 * ks + u][r];
            b[u][r] = rd[2 * ks + u][r];
            inner = __builtin_fmaf(a[u][r], b[u][r], inner);
          }
        const Frag<kW> fs = frag_of<kW>(a[0], a[1]), fd = frag_of<kW>(b[0], b[1]);
        Frag<kIn> f[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) f[i] = lds_frag<kIn, kIn>(lds, i * KD + ks);
        mm_tiles<kW, 0, RT>(ks0, f, fs);
        mm_tiles<kW, 0, RT>(dU, f, fd);
        step();
      }
      {
        f32x4 R[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          ks0[i] *= gate4(gate, C, kEG, rho(i, 4 * lg));
          dU[i] *= gate4(gate, C, kRest, rho(i, 4 * lg));
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            R[i][r] = live ? to_f32(rv[i][r]) - ks0[i][r] : 0.0f;
            dO[i][r] = live ? to_f32(ro[i][r]) : 0.0f;
          }
        }
        static_for<KC>([&](auto kt) {
          const Frag<kW> f = frag_of<kW>(R[2 * kt.value], R[2 * kt.value + 1]);
          Frag<kW> fi[RT];
#pragma unroll
          for (int i = 2 * kt.value; i < RT; ++i) fi[i] = lds_frag<kW, kSW>(inv, lower_frag(i, kt.value));
          mm_tiles<kW, 2 * kt.value, RT>(N, fi, f);
          step();
        });
      }
      // w, before P^T dO joins dU: its rows' sums with those of dN * K S0, and the sum of all
      f32x4 wn[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        wn[i] = gate4(gate, C, kBeta, rho(i, 4 * lg)) * N[i] * dU[i];
        w_sum += (wn[i][0] + wn[i][1]) + (wn[i][2] + wn[i][3]);
      }
      static_for<KC>([&](auto kt) {
        constexpr int to = 2 * kt.value + 2;
        const Frag<kIn> f = frag_of<kIn>(dO[2 * kt.value], dO[2 * kt.value + 1]);
        Frag<kW> fp[RT];
#pragma unroll
        for (int j = 0; j < to; ++j) fp[j] = lds_frag<kW, kSW>(p_t, upper_frag<KC>(j, kt.value));
        mm_tiles<kW, 0, to>(dU, fp, f);
        step();
      });
      static_for<KC>([&](auto kt) {
        constexpr int to = 2 * kt.value + 2;
        const Frag<kW> f = frag_of<kW>(dU[2 * kt.value] * gate4(gate, C, kBeta, rho(2 * kt.value, 4 * lg)),
                                       dU[2 * kt.value + 1] * gate4(gate, C, kBeta, rho(2 * kt.value + 1, 4 * lg)));
        Frag<kW> fi[RT];
#pragma unroll
        for (int j = 0; j < to; ++j) fi[j] = lds_frag<kW, kSW>(inv_t, upper_frag<KC>(j, kt.value));
        mm_tiles<kW, 0, to>(dN, fi, f);
        step();
      });
      // rows t = rho(i, 4 lg + r) of the images lie in lane slots 16 (v / 8) + 4 lg + r of tile i
      char* to_n = lds + oN * 1024 + (col >> 5) * kW * 1024 + (16 * ((col >> 3) & 3) + 4 * lg) * 16 + (col & 7) * 2;
      char* to_dn = to_n + nV * 1024;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float b = row16_tree(dU[i][r] * N[i][r]), m = row16_tree(dN[i][r] * ks0[i][r] + wn[i][r]);
          if (c == 0) {
            red_b[wave][rho(i, r) + 8 * lg] = b;
            red_n[wave][rho(i, r) + 8 * lg] = m;
          }
          __bf16 x[kW], y[kW];
          split<kW>(N[i][r], x);
          split<kW>(dN[i][r], y);
#pragma unroll
          for (int p = 0; p < kW; ++p) {
            *reinterpret_cast<__bf16*>(to_n + (i * KV * kW + p) * 1024 + r * 16) = x[p];
            *reinterpret_cast<__bf16*>(to_dn + (i * KV * kW + p) * 1024 + r * 16) = y[p];
          }
          if (r == 3) step();
        }
      inner = lanes_sum<64>(inner);
      w_sum = lanes_sum<64>(w_sum);
      if (lane == 0) {
        red_s[wave] = inner;
        red_w[wave] = w_sum;
      }
    }
    // the states' rows of this wave's channels, for the last phase
    const int d = rho(wave, c);
    f32x4 xs[KV][2], xd[KV][2];
    if (wave < DT) {
      const float *row_s = ps + static_cast<int64_t>(d < z.dk ? d : 0) * z.dv, *row_d = pd + static_cast<int64_t>(d < z.dk ? d : 0) * z.dv;
      const bool whole = z.dv % 4 == 0;
#pragma unroll
      for (int kv = 0; kv < KV; ++kv)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          xs[kv][u] = load4(row_s, 32 * kv + 8 * lg + 4 * u, z.dv, whole);
          xd[kv][u] = load4(row_d, 32 * kv + 8 * lg + 4 * u, z.dv, whole);
        }
    }
    __syncthreads();

    // dv: eight channels of a token from the image
    for (int id = threadIdx.x; id < C * DV / 8; id += kThreads) {
      const int t = id / (DV / 8), v = id % (DV / 8) * 8;
      const char* from = lds + oDN * 1024 + image_at<KV, kW>(t, v) * 2;
      if (t < n && v < z.dv) {
        f32x4 x{}, y{};
#pragma unroll
        for (int p = kW - 1; p >= 0; --p) {
          const bf16x8 w = *reinterpret_cast<const bf16x8*>(from + p * 1024);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[j] += static_cast<float>(w[j]);
            y[j] += static_cast<float>(w[4 + j]);
          }
        }
        T* to = A.dv.row(t0 + t, h) + v;
        store4(to, z.dv - v, x);
        if (z.dv > v + 4) store4(to + 4, z.dv - v - 4, y);
      }
    }

    // The pair tiles, rows j and columns i: D, P, M, then dP, X and what comes of them.
#pragma unroll 1
    for (int m = 0; m < kMine; ++m) {
      const int p = wave + m * NW;
      if (p >= kPairs) break;
      int i, j;
      pair_of(p, i, j);
      f32x4 qk{}, kk{}, x{}, y{};
      const int row = rho(i, c), at0 = rho(j, 4 * lg);
      const int ti = row < n ? row : n - 1;
      Frag<kIn> fq[KD], fo[KV];
#pragma unroll
      for (int ks = 0; ks < KD; ++ks) fq[ks] = A.q.template frag<kIn>(A.q.from(t0, hk), A.q.lane_off(ti), ks);
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) fo[kv] = A.d_o_rows.template frag<kIn>(A.d_o_rows.from(t0, h), A.d_o_rows.lane_off(ti), kv);
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) mm<kW>(x, lds_frag<kW, kW>(lds + oN * 1024, j * KV + kv), lds_frag<kW, kW>(lds + oDN * 1024, i * KV + kv));
#pragma unroll
      for (int ks = 0; ks < KD; ++ks) {
        const Frag<kIn> kj = lds_frag<kIn, kIn>(lds, j * KD + ks);
        mm<kIn>(kk, kj, lds_frag<kIn, kIn>(lds, i * KD + ks));
        mm<kIn>(qk, kj, fq[ks]);
      }
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) mm<kW>(y, lds_frag<kW, kW>(lds + oN * 1024, j * KV + kv), fo[kv]);
      const f32x4 b = gate4(gate, C, kBeta, at0), hj = gate4(gate, C, kGHi, at0), lj = gate4(gate, C, kGLo, at0);
      const float hi = gate[kGHi * C + row], li = gate[kGLo * C + row];
      f32x4 pd, zz, ev, mx;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int at = at0 + r;
        const bool in = at <= row && row < n, off = at < row && row < n;
        const float dc = in ? decay(hi, li, hj[r], lj[r]) : 0.0f;
        const float dp = in ? b[r] * y[r] * dc * z.scale : 0.0f, bx = off ? x[r] * dc : 0.0f;
        pd[r] = dp;
        zz[r] = -b[r] * bx;
        mx[r] = bx * kk[r];
        ev[r] = dp * qk[r] - b[r] * mx[r];
      }
      // sums over j (rows of the tile) for row i, over i (its columns) for row j
      const Halves s16 = halves16((ev[0] + ev[1]) + (ev[2] + ev[3]));
      const Halves s32 = halves32(s16.a + s16.b);
      if (lg == 0) row_e[i][j][c] = s32.a + s32.b;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float ce = row16_tree(ev[r]), cx = row16_tree(mx[r]);
        if (c == 0) {
          col_e[i][j][4 * lg + r] = ce;
          col_x[i][j][4 * lg + r] = cx;
        }
      }
      // dP * D with rows i and places j, with rows j and places i; Z + Z^T
      char* to_a = img_a + image_at<KC, kW>(row, at0) * 2;
      char* to_b = img_b + image_at<KC, kW>(at0, row) * 2;  // (its rows at0 + r are neighbouring slots)
      const bool diagonal = i / 2 == j / 2;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        __bf16 wp[kW], wz[kW];
        split<kW>(pd[r], wp);
        split<kW>(zz[r], wz);
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          *reinterpret_cast<__bf16*>(to_a + w * 1024 + 2 * r) = wp[w];
          *reinterpret_cast<__bf16*>(to_b + w * 1024 + 16 * r) = wp[w];
          if (!diagonal || at0 + r <= row) {
            *reinterpret_cast<__bf16*>(to_a + 2 * nSq * 1024 + w * 1024 + 2 * r) = wz[w];
            *reinterpret_cast<__bf16*>(to_b + nSq * 1024 + w * 1024 + 16 * r) = wz[w];
          }
        }
      }
    }
    __syncthreads();

    // 16 channels of dq and dk
    if (wave < DT) {
      Frag<kIn> kT[KC], qT[KC], fo[RT], next[RT];
#pragma unroll
      for (int kt = 0; kt < KC; ++kt) {
        const int64_t at = (static_cast<int64_t>(tile) * z.Hk + hk) * (C * DK * kIn);
        kT[kt] = image_frag<kIn, kIn>(A.k_t + at, wave * KC + kt);
        qT[kt] = image_frag<kIn, kIn>(A.q_t + at, wave * KC + kt);
      }
      f32x4 q[RT];
      const uint16_t *po = A.d_o_rows.from(t0, h), *pq = A.q.from(t0, hk) + rho(wave, 0);
      uint32_t off[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int x = rho(i, c), t = x < n ? x : n - 1;
        off[i] = A.d_o_rows.lane_off(t);
        fo[i] = A.d_o_rows.template frag<kIn>(po, off[i], 0);
        q[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = kIn - 1; u >= 0; --u) {
          const bf16x4 w4 = load_at<bf16x4>(pq + u * A.q.words_at, A.q.lane_off(t));
#pragma unroll
          for (int r = 0; r < 4; ++r) q[i][r] += static_cast<float>(w4[r]);
        }
      }
      f32x4 a[RT] = {}, b[RT] = {}, s[RT] = {};
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) {
        if (!full && d >= z.dk)
#pragma unroll
          for (int u = 0; u < 2; ++u) xs[kv][u] = xd[kv][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (kv + 1 < KV)
#pragma unroll
          for (int i = 0; i < RT; ++i)
            next[i] = A.d_o_rows.template frag<kIn>(po, off[i], kv + 1);
        const Frag<kW> fs = frag_of<kW>(xs[kv][0], xs[kv][1]), fd = frag_of<kW>(xd[kv][0], xd[kv][1]);
        Frag<kW> f[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) f[i] = lds_frag<kW, kW>(lds + oDN * 1024, i * KV + kv);
        mm_tiles<kW, 0, RT, true>(b, f, fs);
#pragma unroll
        for (int i = 0; i < RT; ++i) f[i] = lds_frag<kW, kW>(lds + oN * 1024, i * KV + kv);
        mm_tiles<kW, 0, RT, true>(s, f, fd);
        mm_tiles<kW, 0, RT, true>(a, fo, fs);
        if (kv + 1 < KV)
#pragma unroll
          for (int i = 0; i < RT; ++i) fo[i] = next[i];
        step();
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int t = rho(i, c);
        const float eg = gate[kEG * C + t], w = gate[kRest * C + t] * gate[kBeta * C + t];
        a[i] *= eg * z.scale;
        // this wave's part of dO . (scale e^G Q S0) = q . (its part of dq)
        const Halves h16 = halves16((q[i][0] * a[i][0] + q[i][1] * a[i][1]) + (q[i][2] * a[i][2] + q[i][3] * a[i][3]));
        const Halves h32 = halves32(h16.a + h16.b);
        if (lg == 0) red_q[wave][t] = h32.a + h32.b;
        dk[i] += s[i] * w - b[i] * eg;
        dq[i] += a[i];
      }
      static_for<KC>([&](auto kt) {
        constexpr int at = kt.value;
        Frag<kW> f[RT];
#pragma unroll
        for (int i = 2 * at; i < RT; ++i) f[i] = lds_frag<kW, kW>(img_a, i * KC + at);
        mm_tiles<kW, 2 * at, RT, true>(dq, f, kT[at]);
#pragma unroll
        for (int i = 0; i < 2 * at + 2; ++i) f[i] = lds_frag<kW, kW>(img_b, i * KC + at);
        mm_tiles<kW, 0, 2 * at + 2, true>(dk, f, qT[at]);
#pragma unroll
        for (int i = 0; i < RT; ++i) f[i] = lds_frag<kW, kW>(img_c, i * KC + at);
        mm_tiles<kW, 0, RT, true>(dk, f, kT[at]);
        step();
      });
    }
    __syncthreads();

    // dbeta and dg, by the first wave: a lane per token
    if (wave == 0) {
      const int t = lane < C ? lane : 0, rt = rho_tile(t), x = rho_row(t);
      float db = 0.0f, w = 0.0f, dG = 0.0f, inner = 0.0f;
#pragma unroll
      for (int i = 0; i < DV / 16; ++i) {
        db += red_b[i][t];
        w += red_w[i];
        dG -= red_n[i][t];
        inner += red_s[i];
      }
#pragma unroll
      for (int i = 0; i < DT; ++i) dG += red_q[i][t];
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        if (j / 2 <= rt / 2) dG += row_e[rt][j][x];
        if (j / 2 >= rt / 2) {
          dG -= col_e[j][rt][x];
          db -= col_x[j][rt][x];
        }
      }
      // the sums from a row to the end, in float64
      double sum = lane < n ? static_cast<double>(dG) : 0.0;
      if (lane == C - 1) sum += w + static_cast<double>(gate[kEnd * C]) * inner;
#pragma unroll
      for (int o = 1; o < C; o <<= 1) {
        const double other = __shfl_down(sum, o);
        if (lane + o < C) sum += other;
      }
      if (lane < n) {
        const bool cut = A.g[(t0 + t) * A.g_ld + h] < -104.0f;
        A.dg[(t0 + t) * A.dg_ld + h] = from_f32<T>(cut ? 0.0f : static_cast<float>(sum));
        A.dbeta[(t0 + t) * A.dbeta_ld + h] = from_f32<T>(db);
      }
    }
  }
  if (wave_ < DT) {
    const int lane = threadIdx.x & 63, n = static_cast<int>(t1 - t0);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int t = rho(i, lane & 15), d = rho(wave_, 4 * (lane >> 4));
      if (t < n && d < z.dk) {
        store4(A.dq.row(t0 + t, hk) + d, z.dk - d, dq[i]);
        store4(A.dk.row(t0 + t, hk) + d, z.dk - d, dk[i]);
      }
    }
  }
}

template <typename T, int DK>
void launch_chain(const DeltaSizes& z, const ChainArgs<T>& A, hipStream_t st) {
  const int64_t chains = static_cast<int64_t>(z.S) * z.H;
  const int nw = chains >= 256 ? 8 : chains >= 64 ? 4 : 1;  // as in the forward
  const dim3 grid(static_cast<uint32_t>(z.H * ceil_div(z.dv, 16 * nw)), static_cast<uint32_t>(z.S));
  if (nw == 8) hipLaunchKernelGGL((delta_chain_kernel<T, DK, 8>), grid, dim3(512), 0, st, z, A);
  else if (nw == 4) hipLaunchKernelGGL((delta_chain_kernel<T, DK, 4>), grid, dim3(256), 0, st, z, A);
  else hipLaunchKernelGGL((delta_chain_kernel<T, DK, 1>), grid, dim3(64), 0, st, z, A);
}

template <typename T, int DK, int DV>
void launch_grad(const DeltaSizes& z, const GradArgs<T>& A, int dtype, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(delta_tiles(z.T, z.S, dtype)), static_cast<uint32_t>(z.Hk));
  hipLaunchKernelGGL((delta_grad_kernel<T, DK, DV>), grid, dim3(4 * (DK > DV ? DK : DV)), 0, st, z, A);
}

}  // namespace
}  // namespace detgrad

using namespace detgrad;

extern "C" int det_delta_rule_bwd_workspace_size(int64_t T, int64_t S, int64_t Hk, int64_t H, int64_t dk, int64_t dv, int dtype,
                                                 size_t* bytes) {
  if (!bytes) return set_error(DET_ERR_INVALID_ARG, "delta_rule_bwd: bytes is NULL");
  if (int s = delta_check_sizes("delta_rule_bwd", dtype, T, S, Hk, H, dk, dv)) return s;
  const DeltaSizes z{T, (int)S, (int)Hk, (int)H, (int)dk, (int)dv, nullptr, 0.0f};
  *bytes = T == 0 ? 0 : delta_layout(z, dtype, true).all;
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
  const DeltaLayout l = delta_layout(z, dtype, true);
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
  char* base = static_cast<char*>(ws);  // (no tokens: nothing there is read)
  DeltaPrepared r{};
  if (T)
    r = delta_prepare(z, dtype, true, q, q_st, q_sh, k, k_st, k_sh, d_o, do_st, do_sh, g, g_ld, beta, beta_ld, base, l, st);
  const auto words = [&](size_t at) { return reinterpret_cast<const uint16_t*>(base + at); };
  const auto* gate = reinterpret_cast<const float*>(base + l.gates);
  auto* ds = reinterpret_cast<float*>(base + l.ds);
#define DET_DELTA_BWD(E)                                                                                               \
  {                                                                                                                    \
    const Heads<const E> hv{static_cast<const E*>(v), v_st, v_sh}, ho{static_cast<const E*>(d_o), do_st, do_sh};       \
    const ChainArgs<E> A{r.k, ho, words(l.k_t), words(l.q_t), words(l.inverse_t), words(l.p), gate, dfinal_state, ds,  \
                         dinitial_state};                                                                              \
    const GradArgs<E> B{r.k, r.q, r.d_o, hv, ho, {static_cast<E*>(dq), dq_st, dq_sh},                                  \
                        {static_cast<E*>(dk_out), dk_st, dk_sh}, {static_cast<E*>(dv_out), dv_st, dv_sh},              \
                        static_cast<E*>(dg), static_cast<E*>(dbeta), words(l.k_t), words(l.q_t), words(l.inverse),     \
                        words(l.inverse_t), words(l.p), g, gate, states, ds, g_ld, dg_ld, dbeta_ld};                   \
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
