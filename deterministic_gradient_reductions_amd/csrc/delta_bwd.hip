// det_delta_rule_bwd: the gradients of the gated delta rule, in the chunks and with the
// notation of its forward. With A = (I + B M)^-T, dP = lower(dO U^T), X = strict(dN N^T)
// and dS1 the gradient of the state behind the chunk:
//
//   dU = P^T dO + e^(G_C - G) K dS1,   dY = A dU,   dN = B dY,   dV = dN,   dbeta = rowsum(dY * N)
//   dS0 = e^G_C dS1 + scale (e^G Q)^T dO - (e^G K)^T dN
//   dQ = dQ1 + scale (dP * D) K,       dQ1 = scale e^G dO S0^T
//   dK = dK1 - dK0 + scale (dP * D)^T Q + (Z + Z^T) K,   dK1 = e^(G_C - G) U dS1^T,  dK0 = e^G dN S0^T,  Z = -D * X * beta_col
//   dg_t = sum_{i >= t > j} E_ij + sum_{i >= t} (q_i dQ1_i - k_i dK0_i) + sum_{j < t} k_j dK1_j + e^G_C <S0, dS1>,
//          E = dP * P - M * X * beta_col
//
// Every term of dg_t has e^g_t as a factor, since the decays between its two tokens (or states) pass t, so dg keeps its
// digits relative to itself however fast a head forgets. (As the sums from t on of what each row of G takes up, E's
// row sum less its column sum and so on, it is terms without that factor which cancel: what float32 leaves
// of them was more than dg from g of about -8 on.)
//
// Nothing is divided by beta or by a decay. After the forward's preparing kernels (with the
// transposes of P and the inverse) one walks a sequence's chunks backwards as the forward's
// walks them (16 columns of v per wave, dS in registers): it writes dV, every chunk's
// dS1, and dY as an image, as the forward left N. The last kernel takes all chunks side by
// side: in it a wave owns tiles of token pairs first, then 16 channels of dQ and dK;
// the pair matrices change hands in LDS.
//
// 16384 tokens in 8 sequences, 32 heads of 128 x 128, bf16: the chains 440 to 580 us, bound by memory
// (0.97 GB written) while all run and by the longest one after; the last kernel 710 to 800 us for 1.9 GB read.
// There N, dY and dO arrive before the pair tiles and the states' rows under them, and the next head's under
// the last products. (N, dY, the pair matrices and the states in two words, 16 bits, took 560 to 650 us, but 0.3 to 0.4 %
// of dq, dk and dbeta were another bf16 value than the rounded exact one; in three as many as from float32, 0.01 to 0.03 %.)
#include "delta.hpp"

namespace detgrad {
namespace {

template <typename T>
struct ChainArgs {
  Rows k, q;
  Heads<const T> d_o;
  Heads<T> dv;
  const uint16_t* units;
  const float* ds1;
  float *ds, *ds0;  // every chunk's dS1 in blocks, the initial state's gradient
  float* dy;
  int ds_floats;
};

// Workgroups, waves and buffers as in the forward's chain. TEAM: the second wave forms P^T dO
// (a chunk ahead) and scale (e^G Q)^T dO for the first one, and dV and dY's image from what
// that leaves of dY.
template <typename T, int DK, bool TEAM>
__global__ __launch_bounds__(512) void delta_chain_kernel(DeltaSizes z, ChainArgs<T> A) {
  typedef Unit<T, true> Rec;
  constexpr int kIn = DeltaType<T>::kIn, kLogC = DeltaType<T>::kLogC, C = 1 << kLogC;
  constexpr int RT = C / 16, KC = C / 32, DT = DK / 16, KD = DK / 32, kW = kStateWords;
  constexpr int NW = TEAM ? 1 : 8;
  // fragments in LDS: two buffers of K, the inverse and the gates, P and Q; dO of each wave (TEAM: two); what the team hands on
  constexpr int nRows = RT * KD * kIn, nHead = Rec::oP, nP = Rec::nP, nX = 2 * RT + DT;
  constexpr int oP = nRows + nHead, oQ = oP + nP, kBuf = oQ + nRows, oO = 2 * kBuf, oX = oO + (TEAM ? 4 : 2 * NW);
  __shared__ __align__(16) char lds[(oX + (TEAM ? nX : 0)) * 1024];
  const int lane = threadIdx.x & 63, wave_ = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, lg = lane >> 4;
  const int role = TEAM ? wave_ : 0, wave = TEAM ? 0 : wave_;
  const int h = blockIdx.x % z.H, hk = h / (z.H / z.Hk), v0 = ((blockIdx.x / z.H) * NW + wave) * 16, s = blockIdx.y;
  const int dvp = z.dv <= 64 ? 64 : 128;
  const uint32_t lds0 = lds_address(lds);
  char* x = lds + (TEAM ? oX : 0) * 1024;  // dY of these columns
  f32x4 *x_p = lds_tile(x + RT * 1024), *x_q = x_p + RT * 64;  // tiles of P^T dO, of scale (e^G Q)^T dO
  uint32_t r0, r1, first;
  segment_rows(z.offs, s, static_cast<uint32_t>(z.T), kLogC, r0, r1, first);
  const int col = v0 + c, vcol = col < z.dv ? col : z.dv - 1;
  const int chunks = static_cast<int>((r1 - r0 + C - 1) >> kLogC);
  int64_t unit = (static_cast<int64_t>(first) + chunks - 1) * z.H + h;
  int buf = 0;
  const auto o_tile = [&](int buf) { return (oO + 2 * (TEAM ? buf : wave)) * 1024; };
  const bool whole = whole_columns(A.d_o, v0, z.dv);
  T rd[RT][4];
  f32x4 dO[RT];
  const auto start = [&](int ch) { return r0 + (static_cast<uint32_t>(ch) << kLogC); };
  const auto rows_at = [&](int ch) { return r1 - start(ch) < static_cast<uint32_t>(C) ? static_cast<int>(r1 - start(ch)) : C; };
  const auto fetch_do = [&](int ch, int buf) {
    if (whole) fetch_columns<RT>(lds0 + o_tile(buf), A.d_o, start(ch), h, v0, rows_at(ch) - 1);
  };
  const auto load_do = [&](int ch) {
    if (!whole) load_column<RT>(rd, A.d_o.row(start(ch), h), A.d_o.st, vcol, rows_at(ch) - 1);
  };
  const auto take_do = [&](int buf) {
    if (whole) {
      take_columns<RT>(dO, lds + o_tile(buf), static_cast<const T*>(nullptr));
    } else {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) dO[i][r] = to_f32(rd[i][r]);
    }
  };
  const auto fetch_p = [&](int64_t unit, int buf) {
    fetch_image<nP, NW, 5>(lds0 + (buf * kBuf + oP) * 1024, A.units + unit * Rec::kElems + Rec::oP * kFragElems, wave);
  };
  const auto fetch_next = [&](int ch, int64_t unit, int buf) {
    const uint32_t to = lds0 + buf * kBuf * 1024;
    fetch_rows<RT, KD, kIn, NW>(to, A.k, start(ch), rows_at(ch) - 1, hk, wave);
    fetch_image<nHead, NW, 4>(to + nRows * 1024, A.units + unit * Rec::kElems, wave);
    fetch_rows<RT, KD, kIn, NW, 4>(to + oQ * 1024, A.q, start(ch), rows_at(ch) - 1, hk, wave);
  };
  // dU += P^T dO
  const auto add_p = [&](f32x4 (&dU)[RT], const char* img) {
    static_for<KC>([&](auto kt) {
      constexpr int to = 2 * kt.value + 2;
      const Frag<kIn> fo = frag_of<kIn>(dO[2 * kt.value], dO[2 * kt.value + 1]);
      Frag<kW> fp[RT];
#pragma unroll
      for (int j = 0; j < to; ++j) fp[j] = lds_frag<kW, kW>(img, upper_frag<KC>(j, kt.value));
      mm_tiles<kW, 0, to>(dU, fp, fo);
    });
  };
  // S += scale (e^G Q)^T dO
  const auto add_q = [&](f32x4 (&S)[DT], const char* img, const float* gate) {
#pragma unroll
    for (int i = 0; i < RT; ++i) dO[i] *= gate4(gate, C, kEG, rho(i, 4 * lg)) * z.scale;
#pragma unroll
    for (int kt = 0; kt < KC; ++kt) {
      const Frag<kW> fo = frag_of<kW>(dO[2 * kt], dO[2 * kt + 1]);
      Frag<kIn> ft[DT];
#pragma unroll
      for (int i = 0; i < DT; ++i) ft[i] = turned_frag<KD, kIn>(img, i, kt);
      mm_tiles<kW, 0, DT>(S, ft, fo);
    }
  };
  // dV, and dY's image, from dY with rows v and columns t
  const auto put_y = [&](const f32x4 (&yt)[RT], const float* gate, int ch, int64_t unit) {
    put_image<RT>(yt, A.dy + unit * (C * dvp), v0, z.dv, dvp / 32);
    f32x4 dv[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) dv[i] = yt[i] * gate[kBeta * C + rho(i, c)];
    store_rows<RT>(dv, A.dv.row(start(ch), h), A.dv.st, v0, z.dv, rows_at(ch));
  };

  if (role == 2) {
    if (chunks) {
      fetch_next(chunks - 1, unit, 0);
      fetch_p(unit, 0);
      fetch_do(chunks - 1, 0);
    }
    fetch_done();
    __syncthreads();  // the last chunk's fragments are there
    if (chunks > 1) {
      fetch_p(unit - z.H, 1);
      fetch_do(chunks - 2, 1);
    }
    for (int ch = chunks - 1; ch >= 0; --ch, unit -= z.H, buf ^= 1) {
      __syncthreads();  // this chunk's fragments are there, the one's behind it have been read
      if (ch > 0) {
        fetch_next(ch - 1, unit - z.H, buf ^ 1);
        fetch_done_but<2 * nRows + nHead>();  // (the next chunk's P and dO are there)
      }
      __syncthreads();
      if (ch > 1) {  // (this chunk's P and dO have been read)
        fetch_p(unit - 2 * z.H, buf);
        fetch_do(ch - 2, buf);
        if (whole) fetch_done_but<nP + 2>();
        else fetch_done_but<nP>();
      } else {
        fetch_done();
      }
    }
    return;
  }
  if (role == 1) {
    __syncthreads();
    const auto give_p = [&](int buf) {
      f32x4 w[RT] = {};
      add_p(w, lds + (buf * kBuf + oP) * 1024);
#pragma unroll
      for (int i = 0; i < RT; ++i) x_p[i * 64] = w[i];
    };
    if (chunks) {
      load_do(chunks - 1);
      take_do(0);
      give_p(0);
    }
    for (int ch = chunks - 1; ch >= 0; --ch, unit -= z.H, buf ^= 1) {
      lds_read();
      __syncthreads();  // P^T dO is there
      const char* img = lds + buf * kBuf * 1024;
      const float* gate = reinterpret_cast<const float*>(img + (nRows + Rec::oGate) * 1024);
      if (ch > 0) load_do(ch - 1);
      f32x4 w[DT] = {};
      add_q(w, img + oQ * 1024, gate);
#pragma unroll
      for (int i = 0; i < DT; ++i) x_q[i * 64] = w[i];
      lds_read();
      __syncthreads();  // dY is there, and what this wave has left
      f32x4 yt[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) yt[i] = lds_turned(x + i * 1024);
      if (ch > 0) {
        take_do(buf ^ 1);
        give_p(buf ^ 1);
      }
      put_y(yt, gate, ch, unit);
    }
    return;
  }

  const int64_t size = static_cast<int64_t>(z.dk) * z.dv, of = (static_cast<int64_t>(s) * z.H + h) * size;
  f32x4 S[DT] = {};
  if (A.ds1) {
    float y[DT][4];
    load_state<DT>(y, A.ds1 + of, z.dk, z.dv, vcol);
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = rho(i, 4 * lg + r) < z.dk ? y[i][r] : 0.0f;
  }
  Frag<kW> f[KD];  // of S
#pragma unroll
  for (int ks = 0; ks < KD; ++ks) f[ks] = frag_of<kW>(S[2 * ks], S[2 * ks + 1]);
  if (TEAM) {
    __syncthreads();
  } else {
    if (chunks) {
      load_do(chunks - 1);
      fetch_do(chunks - 1, 0);
      fetch_next(chunks - 1, unit, 0);
      fetch_p(unit, 0);
    }
    fetch_done();
  }
  for (int ch = chunks - 1; ch >= 0; --ch, unit -= z.H, buf ^= 1) {
    __syncthreads();  // this chunk's fragments are there, the last one's have been read
    if (!TEAM) {
      if (ch > 0) {
        fetch_next(ch - 1, unit - z.H, buf ^ 1);
        fetch_p(unit - z.H, buf ^ 1);
      }
      take_do(0);
    }
    if (v0 < z.dv) {
      if (!TEAM) lds_read();
      store_block<DT>(S, A.ds + unit * A.ds_floats + v0 * z.dk, z.dk, TEAM ? x : lds + o_tile(0));
    }
    const char* img = lds + buf * kBuf * 1024;
    const float* gate = reinterpret_cast<const float*>(img + (nRows + Rec::oGate) * 1024);
    f32x4 dU[RT] = {};
#pragma unroll
    for (int ks = 0; ks < KD; ++ks) {
      Frag<kIn> fk[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) fk[i] = row_frag<kIn>(img, i * KD + ks);
      mm_tiles<kW, 0, RT>(dU, fk, f[ks]);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) dU[i] *= gate4(gate, C, kRest, rho(i, 4 * lg));
    if (TEAM) {
#pragma unroll
      for (int i = 0; i < RT; ++i) dU[i] += x_p[i * 64];
    } else {
      f32x4 w[RT] = {};  // (summed by itself, as the team does)
      add_p(w, img + oP * 1024);
#pragma unroll
      for (int i = 0; i < RT; ++i) dU[i] += w[i];
    }
    f32x4 dN[RT] = {};  // dY
    static_for<KC>([&](auto kt) {
      constexpr int to = 2 * kt.value + 2;
      const Frag<kW> fu = frag_of<kW>(dU[2 * kt.value], dU[2 * kt.value + 1]);
      Frag<kW> fi[RT];
#pragma unroll
      for (int j = 0; j < to; ++j) fi[j] = lds_frag<kW, kW>(img + nRows * 1024, upper_frag<KC>(j, kt.value));
      mm_tiles<kW, 0, to>(dN, fi, fu);
    });
    const float el = gate[kEnd * C];
    if (TEAM) {
#pragma unroll
      for (int i = 0; i < RT; ++i) *lds_tile(x + i * 1024) = dN[i];
    } else {
      f32x4 yt[RT];
      lds_read();
      turn_tiles<RT>(yt, dN, lds + o_tile(0));
      put_y(yt, gate, ch, unit);
      if (ch > 0) {
        lds_read();
        load_do(ch - 1);
        fetch_do(ch - 1, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) dN[i] *= gate4(gate, C, kEGBeta, rho(i, 4 * lg));
    Frag<kW> fn[KC];
#pragma unroll
    for (int kt = 0; kt < KC; ++kt) fn[kt] = frag_of<kW>(dN[2 * kt], dN[2 * kt + 1]);
#pragma unroll
    for (int i = 0; i < DT; ++i) S[i] *= el;
    if (TEAM) {
      __syncthreads();  // the second wave's part of dS is there
#pragma unroll
      for (int i = 0; i < DT; ++i) S[i] += x_q[i * 64];
    } else {
      f32x4 w[DT] = {};
      add_q(w, img + oQ * 1024, gate);
#pragma unroll
      for (int i = 0; i < DT; ++i) S[i] += w[i];
    }
    next_state<kIn, KC>(S, f, img, fn, 1.0f);
    if (!TEAM) fetch_done();
  }
  if (A.ds0) store_state<DT>(S, A.ds0 + of, z.dk, z.dv, col);
}

template <typename T>
struct GradArgs {
  Rows k, q, d_o;
  Heads<T> dq, dk;
  T *dg, *dbeta;
  const uint16_t* units;
  const float *dy, *saved, *ds;
  int64_t dg_ld, dbeta_ld;
  int image_floats, saved_floats, ds_floats;
};

// No instruction is moved over this: what a step loads is not loaded steps before, in
// registers that the steps between need.
__device__ __forceinline__ void step() { __builtin_amdgcn_sched_barrier(0); }

// Pair tile p: tiles i of rows and j of columns of the lower triangle, whole blocks of 32.
__device__ __forceinline__ void pair_of(int p, int& i, int& j) {
  i = p < 4 ? p >> 1 : 2 + ((p - 4) >> 2);
  j = p < 4 ? p & 1 : (p - 4) & 3;
}

// Workgroup (tile, hk): one chunk of one key head, its value heads in turn. K, Q and dO come to LDS past the
// registers, the states' rows into registers meanwhile. N and dY are float32 in memory (two thirds of their words) and
// pass the registers, where each of their fragments becomes words once, under the last products of the head before.
//
// For a bf16 call's 128 channels of v LDS has no room for the pair matrices beside N, dY and dO. There (kShare) they wait
// in registers and take the place of dY, whose next one waits in registers for them.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(4 * (DK > DV ? DK : DV)) void delta_grad_kernel(DeltaSizes z, GradArgs<T> A) {
  constexpr int kIn = DeltaType<T>::kIn, kW = kStateWords, kLogC = DeltaType<T>::kLogC, C = 1 << kLogC;
  constexpr int NW = (DK > DV ? DK : DV) / 16, RT = C / 16, KC = C / 32, DT = DK / 16, KD = DK / 32, KV = DV / 32;
  constexpr int kFrags = KC * (KC + 1), kPairs = 2 * kFrags, kMine = (kPairs + NW - 1) / NW;  // pair tiles, of a wave
  // 1024-byte fragments of the images
  constexpr int nK = RT * KD * kIn, nO = RT * KV * kIn, nV = RT * KV * kW, nTri = kFrags * kW,
                nGate = Unit<T, true>::nGate;
  constexpr bool kShare = 2 * nK + nO + 2 * nV + 2 * nTri + 2 * nGate > 148;
  constexpr int oQ = nK, oN = 2 * nK, oO = oN + nV, oY = oO + nO, oA = kShare ? oY : oY + nV, oZ = oA + nTri,
                oGate = kShare ? oY + nV : oZ + nTri;
  static_assert(2 * nTri <= nV || !kShare, "the pair matrices in dY's place");
  constexpr int nF = RT * KV, kEach = (nF + NW - 1) / NW;  // fragments of N and of dY, of a wave
  __shared__ __align__(16) char lds[(oGate + 2 * nGate) * 1024];
  __shared__ float red_q[NW][C], red_w[NW][C], red_s[NW], diag[C];
  // E's sums over four columns j from 4 m on, per row (padded: rows start on banks of their own); its crossing sums with
  // j in t's own four, per row tile; and with j before them
  constexpr int kRuns = C / 4, kRunLd = kRuns + 4;
  __shared__ __align__(16) float run_e[C][kRunLd], near_e[RT][C], far_e[C];
  char *img_a = lds + oA * 1024, *img_z = lds + oZ * 1024;
  const uint32_t lds0 = lds_address(lds);
  const int wave_ = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = blockIdx.x;
  const int hk = blockIdx.y, group = z.H / z.Hk;
  int e;
  uint32_t t0, t1, s0, s1;
  if (!segment_tile<1>(z.offs, z.S, static_cast<uint32_t>(z.T), kLogC, tile, e, t0, t1, s0, s1)) return;
  f32x4 dq[RT] = {}, dk[RT] = {};  // rows d, columns t
  f32x4 qk[kMine], kk[kMine];      // of this wave's pair tiles
  f32x4 xs[KV][2], xd[KV][2];      // the states' rows of this wave's channels
  typedef f32x4 Mine[kEach][2];  // this wave's fragments of N or dY
  const auto fetch_head = [&](int h, Mine& rn, Mine& ry) {
    const int wave = here(wave_), n = here(static_cast<int>(t1 - t0)), buf = (h - hk * group) & 1;
    const uint32_t at = static_cast<uint32_t>(here_lane(threadIdx.x) & 63) * 16u;
    const int64_t unit = static_cast<int64_t>(tile) * z.H + h;
    const float *pn = A.saved + unit * A.saved_floats, *py = A.dy + unit * (nF * kFragFloats);
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int f = wave + u * NW;
      if (nF % NW && f >= nF) continue;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        rn[u][e] = load_at<f32x4>(pn + f * kFragFloats + e * 256, at);
        ry[u][e] = load_at<f32x4>(py + f * kFragFloats + e * 256, at);
      }
    }
    fetch_rows<RT, KV, kIn, NW>(lds0 + oO * 1024, A.d_o, t0, n - 1, h, wave);
    fetch_image<nGate, NW, 7>(lds0 + (oGate + buf * nGate) * 1024, A.units + unit * Unit<T, true>::kElems + Unit<T, true>::oGate * kFragElems, wave);
  };
  const auto put_words = [&](int at, const Mine& x) {
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int f = here(wave_) + u * NW;
      if (nF % NW && f >= nF) continue;
      lds_put<kW>(lds + at * 1024, f, frag_of<kW>(x[u][0], x[u][1]));
    }
  };
  const auto load_states = [&](int h) {
    const int wave = here(wave_), lane = here_lane(threadIdx.x) & 63, c = lane & 15, lg = lane >> 4;
    if (DT != NW && wave >= DT) return;
    const int64_t unit = static_cast<int64_t>(tile) * z.H + h;
    const float *ps = A.saved + unit * A.saved_floats + A.image_floats, *pd = A.ds + unit * A.ds_floats;
    const int d = rho(wave, c);
    // (every load stays in its block; what lies behind dk or dv is masked below)
#pragma unroll
    for (int kv = 0; kv < KV; ++kv) {
      const int block = 2 * kv + (lg >> 1);
      const uint32_t off = static_cast<uint32_t>(((16 * block < z.dv ? block : 0) * z.dk + (d < z.dk ? d : 0)) * 16 + 8 * (lg & 1)) * 4u;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        xs[kv][u] = load_at<f32x4>(ps + 4 * u, off);
        xd[kv][u] = load_at<f32x4>(pd + 4 * u, off);
      }
    }
  };
  // dP * D and Z of a pair tile as images of rows i and places j: row tile i, row c, places 4 lg .. of fragment j / 2
  const auto put_pairs = [&](int i, int j, const f32x4& ps, const f32x4& pz) {
    const int to = lower_frag(i, j >> 1) * kW * 1024 + row_place() * 16 + (j & 1) * 8;
    uint32_t w0[kW], w1[kW], w2[kW], w3[kW];
    split2<kW>(ps[0], ps[1], w0);
    split2<kW>(ps[2], ps[3], w1);
    split2<kW>(pz[0], pz[1], w2);
    split2<kW>(pz[2], pz[3], w3);
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      *reinterpret_cast<uint64_t*>(img_a + to + w * 1024) = w0[w] | static_cast<uint64_t>(w1[w]) << 32;
      *reinterpret_cast<uint64_t*>(img_z + to + w * 1024) = w2[w] | static_cast<uint64_t>(w3[w]) << 32;
    }
  };
  const int h0 = hk * group;
  fetch_rows<RT, KD, kIn, NW>(lds0, A.k, t0, static_cast<int>(t1 - t0) - 1, hk, wave_);
  fetch_rows<RT, KD, kIn, NW, 4>(lds0 + oQ * 1024, A.q, t0, static_cast<int>(t1 - t0) - 1, hk, wave_);
  {
    Mine rn, ry;
    fetch_head(h0, rn, ry);
    put_words(oN, rn);
    put_words(oY, ry);
  }

  for (int h = h0; h < h0 + group; ++h) {
    const int wave = here(wave_), lane = here_lane(threadIdx.x) & 63, c = lane & 15, lg = lane >> 4;
    const int n = here(static_cast<int>(t1 - t0)), d = rho(wave, c);
    const float* gate = reinterpret_cast<const float*>(lds + (oGate + ((h - h0) & 1) * nGate) * 1024);
    const bool more = h + 1 < h0 + group;
    load_states(h);
    if (DT == NW || wave < DT) fetch_done_but<4 * KV>();  // (the states' rows are still on their way)
    else fetch_done();
    __syncthreads();

    // The pair tiles, rows j and columns i: D, P, M, then dP, X and what comes of them.
    f32x4 pd[kMine], zz[kMine];
    static_for<kMine>([&](auto mine) {
      constexpr int m = mine.value;
      const int p = wave + m * NW;
      if (p >= kPairs) return;
      int i, j;
      pair_of(p, i, j);
      f32x4 x{}, y{};
      const int row = rho(i, c), at0 = rho(j, 4 * lg);
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) {
        const Frag<kW> f = lds_frag<kW, kW>(lds + oN * 1024, j * KV + kv);
        mm<kW>(x, f, lds_frag<kW, kW>(lds + oY * 1024, i * KV + kv));
        mm<kW>(y, f, row_frag<kIn>(lds + oO * 1024, i * KV + kv));
      }
      if (h == h0) {
        qk[m] = kk[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = 0; ks < KD; ++ks) {
          const Frag<kIn> kj = row_frag<kIn>(lds, j * KD + ks);
          mm<kIn>(kk[m], kj, row_frag<kIn>(lds, i * KD + ks));
          mm<kIn>(qk[m], kj, row_frag<kIn>(lds + oQ * 1024, i * KD + ks));
        }
      }
      const f32x4 b = gate4(gate, C, kBeta, at0), hj = gate4(gate, C, kGHi, at0), lj = gate4(gate, C, kGLo, at0);
      const float hi = gate[kGHi * C + row], li = gate[kGLo * C + row], bi = gate[kBeta * C + row];
      f32x4 ps, pz, ev;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int at = at0 + r;
        if (at == row) diag[row] = x[r];  // dY . N of one token
        const bool in = at <= row && row < n, off = at < row && row < n;
        const float dc = in ? decay(hi, li, hj[r], lj[r]) : 0.0f;
        const float dp = in ? b[r] * y[r] * dc * z.scale : 0.0f, bx = off ? b[r] * bi * x[r] * dc : 0.0f;
        ps[r] = dp;
        pz[r] = -bx;
        ev[r] = off ? dp * qk[m][r] - bx * kk[m][r] : 0.0f;  // (no token's pair with itself crosses a t)
      }
      // a lane's four columns j are one run: t behind them takes them all, t among them those before it
      run_e[row][at0 >> 2] = (ev[0] + ev[1]) + (ev[2] + ev[3]);
      float before = ev[0];
#pragma unroll
      for (int r = 1; r < 4; ++r) {
        const float ne = row16_tree(row >= at0 + r ? before : 0.0f);
        if (c == 0) near_e[i][at0 + r] = ne;
        before += ev[r];
      }
      if (kShare) {
        pd[m] = ps;
        zz[m] = pz;
      } else {
        put_pairs(i, j, ps, pz);
      }
    });

    // 16 channels of dq and dk
    if (DT == NW || wave < DT) {
      f32x4 a[RT] = {}, b[RT] = {}, s[RT] = {};
      float inner = 0.0f;
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool in = d < z.dk && 32 * kv + 8 * lg + 4 * u + r < z.dv;
            xs[kv][u][r] = in ? xs[kv][u][r] : 0.0f;
            xd[kv][u][r] = in ? xd[kv][u][r] : 0.0f;
            inner = __builtin_fmaf(xs[kv][u][r], xd[kv][u][r], inner);
          }
        const Frag<kW> fd = frag_of<kW>(xd[kv][0], xd[kv][1]);
        Frag<kW> f[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) f[i] = lds_frag<kW, kW>(lds + oN * 1024, i * KV + kv);
        mm_tiles<kW, 0, RT, true>(s, f, fd);
        step();
      }
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) {
        const Frag<kW> fs = frag_of<kW>(xs[kv][0], xs[kv][1]);
        Frag<kW> f[RT];
        Frag<kIn> fo[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) f[i] = lds_frag<kW, kW>(lds + oY * 1024, i * KV + kv);
        mm_tiles<kW, 0, RT, true>(b, f, fs);
#pragma unroll
        for (int i = 0; i < RT; ++i) fo[i] = row_frag<kIn>(lds + oO * 1024, i * KV + kv);
        mm_tiles<kW, 0, RT, true>(a, fo, fs);
        step();
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int t = rho(i, c);
        const float eg = gate[kEG * C + t], bt = gate[kBeta * C + t];
        a[i] *= eg * z.scale;
        b[i] *= eg * bt;
        s[i] *= gate[kRest * C + t] * bt;
        f32x4 q{}, k{};
#pragma unroll
        for (int u = kIn - 1; u >= 0; --u) {
          const char* row = lds + ((i * KD + (wave >> 1)) * kIn + u) * 1024 + row_place() * 16 + (wave & 1) * 8;
          const bf16x4 wk = *reinterpret_cast<const bf16x4*>(row), wq = *reinterpret_cast<const bf16x4*>(row + oQ * 1024);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            q[r] += static_cast<float>(wq[r]);
            k[r] += static_cast<float>(wk[r]);
          }
        }
        // this wave's part of Q * dQ1 - K * dK0 and of K * dK1 (tokens past the end: K stands for another's, but a, b, s are 0)
        float dot = 0.0f, dot_w = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          dot_w = __builtin_fmaf(k[r], s[i][r], dot_w);
          dot += __builtin_fmaf(q[r], a[i][r], -(k[r] * b[i][r]));
        }
        const Halves h16 = halves16(dot), w16 = halves16(dot_w);
        const Halves h32 = halves32(h16.a + h16.b), w32 = halves32(w16.a + w16.b);
        if (lg == 0) {
          red_q[wave][t] = h32.a + h32.b;
          red_w[wave][t] = w32.a + w32.b;
        }
        dk[i] += s[i] - b[i];
        dq[i] += a[i];
      }
      inner = lanes_sum<64>(inner);
      if (lane == 0) red_s[wave] = inner;
    }

    __syncthreads();  // N, dY and dO have been read
    Mine rn = {}, ry = {};  // (no values of the head before, which would stay in registers all the way)
    if (more) fetch_head(h + 1, rn, ry);
    if constexpr (kShare) {
      static_for<kMine>([&](auto mine) {
        constexpr int m = mine.value;
        const int p = wave + m * NW;
        if (p >= kPairs) return;
        int i, j;
        pair_of(p, i, j);
        put_pairs(i, j, pd[m], zz[m]);
      });
      __syncthreads();  // the pair matrices are there
    }

    // E's crossing sums for the t of a run, a lane per row i: its runs before that one, summed over the rows from t on
    for (int m = wave; m < kRuns; m += NW) {
      float p = 0.0f;
#pragma unroll
      for (int u = 0; u < kRuns; u += 4) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(&run_e[lane & (C - 1)][u]);
#pragma unroll
        for (int r = 0; r < 4; ++r) p += u + r < m ? w[r] : 0.0f;
      }
      f32x4 t;
      t[3] = lanes_sum<64>(lane >= 4 * m + 4 && lane < C ? p : 0.0f);
#pragma unroll
      for (int r = 3; r >= 0; --r) t[r] = (r < 3 ? t[r + 1] : t[3]) + readlane(p, 4 * m + r);
      if (lane == 0) *reinterpret_cast<f32x4*>(&far_e[4 * m]) = t;
    }

    if (DT == NW || wave < DT) {
      static_for<KC>([&](auto kt) {
        constexpr int at = kt.value;
        const Frag<kIn> kT = turned_frag<KD, kIn>(lds, wave, at), qT = turned_frag<KD, kIn>(lds + oQ * 1024, wave, at);
        Frag<kW> f[RT];
#pragma unroll
        for (int i = 2 * at; i < RT; ++i) f[i] = row_frag<kW>(img_a, lower_frag(i, at));
        mm_tiles<kW, 2 * at, RT, true>(dq, f, kT);
#pragma unroll
        for (int i = 2 * at; i < RT; ++i) f[i] = row_frag<kW>(img_z, lower_frag(i, at));
        mm_tiles<kW, 2 * at, RT, true>(dk, f, kT);
        step();
#pragma unroll
        for (int j = 0; j < 2 * at + 2; ++j) f[j] = turned_frag<kW>(img_a, j, lower_frag(2 * at, j >> 1), lower_frag(2 * at + 1, j >> 1));
        mm_tiles<kW, 0, 2 * at + 2, true>(dk, f, qT);
#pragma unroll
        for (int j = 0; j < 2 * at + 2; ++j) f[j] = turned_frag<kW>(img_z, j, lower_frag(2 * at, j >> 1), lower_frag(2 * at + 1, j >> 1));
        mm_tiles<kW, 0, 2 * at + 2, true>(dk, f, kT);
        step();
      });
    }
    if (more) {
      put_words(oN, rn);
      if (!kShare) put_words(oY, ry);
    }
    __syncthreads();
    if (kShare && more) put_words(oY, ry);

    // dbeta and dg, by the first wave: a lane per token
    if (wave == 0) {
      const int t = lane < C ? lane : 0, rt = rho_tile(t);
      float q = 0.0f, w = 0.0f, inner = 0.0f, ce = far_e[t];
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        q += red_q[i][t];
        w += red_w[i][t];
        inner += red_s[i];
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
        if (i / 2 >= rt / 2 && (t & 3)) ce += near_e[i][t];
      // the rows' sums from t to the end, and those before t (taking a row off a sum with it would not leave them), in float64
      const float w0 = __shfl_up(w, 1);
      double from = lane < n ? static_cast<double>(q) : 0.0, to = lane > 0 && lane < n ? static_cast<double>(w0) : 0.0;
#pragma unroll
      for (int o = 1; o < C; o <<= 1) {
        const double f = __shfl_down(from, o), g = __shfl_up(to, o);
        if (lane + o < C) from += f;
        if (lane >= o) to += g;
      }
      if (lane < n) {
        const double dg = from + to + ce + static_cast<double>(gate[kEnd * C]) * inner;
        A.dg[(t0 + t) * A.dg_ld + h] = from_f32<T>(static_cast<float>(dg));
        A.dbeta[(t0 + t) * A.dbeta_ld + h] = from_f32<T>(diag[t]);
      }
    }
  }
  if (DT == NW || wave_ < DT) {
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
  const bool teams = delta_teams(z);
  const dim3 grid(static_cast<uint32_t>(z.H * (teams ? delta_pad(z.dv) / 16 : 1)), static_cast<uint32_t>(z.S));
  if (teams) hipLaunchKernelGGL((delta_chain_kernel<T, DK, true>), grid, dim3(192), 0, st, z, A);
  else hipLaunchKernelGGL((delta_chain_kernel<T, DK, false>), grid, dim3(512), 0, st, z, A);
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
                     {"states", range1d(states, delta_tiles(T, S, dtype) * H * delta_saved_floats(dk, dv, dtype) * 4), 16},
                     {"dfinal_state", range1d(dfinal_state, S * state)}};
  if (int s = check_buffers(what, outs, 7, ins, 9)) return s;
  const hipStream_t st = as_stream(stream);
  char* base = static_cast<char*>(ws);  // (no tokens: nothing there is read)
  DeltaPrepared r{};
  if (T)
    r = delta_prepare(z, dtype, true, q, q_st, q_sh, k, k_st, k_sh, d_o, do_st, do_sh, g, g_ld, beta, beta_ld, base, l, st);
  const auto words = [&](size_t at) { return reinterpret_cast<uint16_t*>(base + at); };
  auto* ds = reinterpret_cast<float*>(base + l.ds);
  const int image = static_cast<int>(delta_image_floats(dv, dtype)), saved = static_cast<int>(delta_saved_floats(dk, dv, dtype)),
            block = static_cast<int>(delta_block_floats(dk, dv));
#define DET_DELTA_BWD(E)                                                                                               \
  {                                                                                                                    \
    const ChainArgs<E> A{r.k, r.q, {static_cast<const E*>(d_o), do_st, do_sh},                                         \
                         {static_cast<E*>(dv_out), dv_st, dv_sh}, words(l.units), dfinal_state, ds, dinitial_state,    \
                         reinterpret_cast<float*>(base + l.dy), block};                                                \
    const GradArgs<E> B{r.k, r.q, r.d_o, {static_cast<E*>(dq), dq_st, dq_sh},                                          \
                        {static_cast<E*>(dk_out), dk_st, dk_sh}, static_cast<E*>(dg), static_cast<E*>(dbeta),          \
                        words(l.units), reinterpret_cast<const float*>(base + l.dy), states, ds, dg_ld, dbeta_ld,      \
                        image, saved, block};                                                                          \
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
