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
// Two or three kernels. One copies K and Q into padded bf16 words where they are not
// bf16 in whole 16-byte rows already. One forms, for all chunks side by side, P and the
// inverse of I + M B (a wave per chunk and head: 16 x 16 diagonal blocks by substitution, the
// blocks below by float32 matrix instructions) and leaves both as fragments. The last walks the
// chunks of one sequence and value head in order. There a wave owns 16 columns of v, so its
// part of S, N, U and O depends on no other wave, what one product leaves in its registers is
// the next one's operand, and the other operands are fragments of 16 bytes per lane,
// shared by the workgroup through LDS. What is not on the chain of states is formed
// before it.
//
// 32768 tokens of one sequence, 32 heads of 128 x 128, bf16: 1301 us, most of it the chains, 2.2 us a chunk, of which the
// 132 matrix instructions of the wave that carries the state are 0.9 us. Under a profiler, whose passes are slower (1434 us
// in all): 214 us for P and the inverses (0.27 GB read and 0.64 GB written) and 1221 us for the chains. There, too, 16384
// tokens of 8 sequences with what the backward needs take 127 and 450 to 640 us, by the longest (0.97 GB written).
#include "delta.hpp"

namespace detgrad {
namespace {

// ------------------------------------------------------------------------------- copy
// Up to three tensors of a call that the kernels cannot read as they are.
template <typename T>
struct Copies {
  Heads<const T> x[3];
  uint16_t* rows[3];
  int heads[3], dim[3], pad[3], n;
};
// Workgroup (tile, head, tensor): the chunk's rows in padded words. (One launch for all of them: a
// launch is 6 us where there is little to copy.)
template <typename T>
__global__ __launch_bounds__(256) void delta_copy_kernel(DeltaSizes z, Copies<T> A) {
  constexpr int kIn = DeltaType<T>::kIn, kLogC = DeltaType<T>::kLogC, C = 1 << kLogC, kEach = 2;
  const uint32_t tile = blockIdx.x;
  const int h = blockIdx.y, heads = A.heads[blockIdx.z], dim = A.dim[blockIdx.z], pad = A.pad[blockIdx.z];
  const Heads<const T> x = A.x[blockIdx.z];
  uint16_t* rows = A.rows[blockIdx.z];
  int e;
  uint32_t r0, r1, s0, s1;
  if (h >= heads || !segment_tile<1>(z.offs, z.S, static_cast<uint32_t>(z.T), kLogC, tile, e, r0, r1, s0, s1)) return;
  const int n = static_cast<int>(r1 - r0), log_row = pad == 64 ? 4 : 5;  // of groups of four channels
  const bool whole = dim % 4 == 0;
  for (int id0 = threadIdx.x; id0 < C << log_row; id0 += kEach * 256) {
    f32x4 v[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int t = (id0 + u * 256) >> log_row, d = 4 * ((id0 + u * 256) & ((1 << log_row) - 1));
      v[u] = load4(x.row(r0 + (t < n ? t : 0), h), d, dim, whole);
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int t = (id0 + u * 256) >> log_row, d = 4 * ((id0 + u * 256) & ((1 << log_row) - 1));
      if (t >= n) continue;
      uint32_t a[kIn], b[kIn];
      split2<kIn>(v[u][0], v[u][1], a);
      split2<kIn>(v[u][2], v[u][3], b);
#pragma unroll
      for (int p = 0; p < kIn; ++p) {
        const uint64_t w = a[p] | static_cast<uint64_t>(b[p]) << 32;
        __builtin_memcpy(rows + ((static_cast<int64_t>(r0 + t) * heads + h) * kIn + p) * pad + d, &w, 8);
      }
    }
  }
}

// ------------------------------------------------------------- inverse, P and gates
constexpr int kPrepWaves = 4;

// The inverse of I + M B and P as images of rows i and places j; BWD: that of I + B M and P
// transposed (rows j, places i), P in the words of the states too.
template <typename T, int DK, bool BWD>
__global__ __launch_bounds__(64 * kPrepWaves, 2) void delta_prep_kernel(DeltaSizes z, Rows k, Rows q,
                                                                     const float* __restrict__ g, int64_t g_ld,
                                                                     const T* __restrict__ beta, int64_t beta_ld,
                                                                     uint16_t* __restrict__ out, int64_t units) {
  constexpr int kIn = DeltaType<T>::kIn, kLogC = DeltaType<T>::kLogC, C = 1 << kLogC, RT = C / 16, KC = C / 32, KS = DK / 32;
  typedef Unit<T, BWD> Rec;
  constexpr int kW = kStateWords;
  constexpr int kLd = C + 4;  // 16-byte rows whose starts move through the banks
  __shared__ __align__(16) float lds[kPrepWaves][C * kLd + 3 * C];
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
  out += unit * Rec::kElems;
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
    const float eg = exp_e(h0) * (1.0f + h1), end = __shfl(eg, C - 1);
    float* to = reinterpret_cast<float*>(out + Rec::oGate * kFragElems);
    if (lane < C) {
      hi[lane] = h0;
      lo[lane] = h1;
      be[lane] = b;
      to[kGHi * C + lane] = h0;
      to[kGLo * C + lane] = h1;
      to[kEG * C + lane] = lane < n ? eg : 0.0f;
      const double rest = last - G;
      const float q0 = static_cast<float>(rest);
      const float er = exp_e(q0) * (1.0f + static_cast<float>(rest - q0));
      to[kRest * C + lane] = er;
      to[kRestBeta * C + lane] = er * b;
      to[kEGBeta * C + lane] = -eg * b;
      to[kBeta * C + lane] = b;
      to[kEnd * C + lane] = end;
    }
  }
  wave_fence();

  // K K^T and Q K^T: rows j and columns i (BWD: rows i and columns j)
  f32x4 kk[RT][RT] = {}, qk[RT][RT] = {};
  {
    const uint16_t *pk = k.from(r0, hk), *pq = q.from(r0, hk);
    uint32_t ok[RT], oq[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int t = rho(i, c), row = t < n ? t : n - 1;
      ok[i] = k.lane_off(row);
      oq[i] = q.lane_off(row);
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      Frag<kIn> fk[RT], fq[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        fk[i] = k.frag<kIn>(pk, ok[i], ks);
        fq[i] = q.frag<kIn>(pq, oq[i], ks);
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < RT && j / 2 <= i / 2; ++j) {
          if (BWD) {
            mm<kIn>(kk[i][j], fk[i], fk[j]);
            mm<kIn>(qk[i][j], fq[i], fk[j]);
          } else {
            mm<kIn>(kk[i][j], fk[j], fk[i]);
            mm<kIn>(qk[i][j], fk[j], fq[i]);
          }
        }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < RT && j / 2 <= i / 2; ++j) {
      const int col = rho(BWD ? j : i, c), row0 = rho(BWD ? i : j, 4 * lg);
      const float hc = hi[col], lc = lo[col];
      f32x4 m;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = row0 + r, ti = BWD ? row : col, tj = BWD ? col : row;
        const float d = BWD ? decay(hi[row], lo[row], hc, lc) : decay(hc, lc, hi[row], lo[row]);
        m[r] = tj < ti ? kk[i][j][r] * d * be[row] : 0.0f;  // beta of j, BWD: of i
        qk[i][j][r] = tj <= ti && ti < n ? qk[i][j][r] * d * z.scale : 0.0f;
      }
      if (BWD) {
#pragma unroll
        for (int r = 0; r < 4; ++r) a[(row0 + r) * kLd + col] = m[r];
      } else {
        *reinterpret_cast<f32x4*>(a + col * kLd + row0) = m;
      }
    }
  {
    uint16_t* to = out + Rec::oP * kFragElems;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int m = 0; m < KC; ++m) {
        if (BWD && m >= i / 2) image_put<kW>(to, upper_frag<KC>(i, m), frag_of<kW>(qk[2 * m][i], qk[2 * m + 1][i]));
        if (!BWD && m <= i / 2) image_put<kW>(to, lower_frag(i, m), frag_of<kW>(qk[i][2 * m], qk[i][2 * m + 1]));
      }
  }
  wave_fence();

  // The inverses of the diagonal blocks: lane group lg takes block lg, lane c its
  // column c, by substitution down the rows.
  {
    float x[16];
    const int blk = lg < RT ? lg : 0;
    const float* p = a + (16 * blk) * kLd + 16 * blk;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float s = r == c ? 1.0f : 0.0f;
#pragma unroll
      for (int m = 0; m < r; m += 4) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(p + r * kLd + m);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (m + u < r) s = __builtin_fmaf(-w[u], x[m + u], s);
      }
      x[r] = s;
    }
    wave_fence();
    if (lg < RT)
#pragma unroll
      for (int r = 0; r < 16; ++r) a[(16 * blk + r) * kLd + 16 * blk + c] = x[r];
    // above the diagonal inside the fragments of 32 places
#pragma unroll
    for (int m = 0; m < KC; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) a[(32 * m + 4 * lg + r) * kLd + 32 * m + 16 + c] = 0.0f;
  }
  wave_fence();

  // The blocks below, column by column of blocks: X_ij = -X_ii sum_{j <= m < i} (M B)_im X_mj.
  // Float32 matrix instructions; the place 4 lg + s of the sum is step s of lane group
  // lg. A column of blocks is read no more once it is done, and X takes its place.
  const auto row4 = [&](int i, int j) { return *reinterpret_cast<const f32x4*>(a + (16 * i + c) * kLd + 16 * j + 4 * lg); };
#pragma unroll
  for (int j = 0; j < RT - 1; ++j) {
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
    wave_fence();
#pragma unroll
    for (int i = j + 1; i < RT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) a[(16 * i + 4 * lg + r) * kLd + 16 * j + c] = X[i][r];
  }
  wave_fence();
  uint16_t* to = out;
  if (!BWD) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int m = 0; m <= i / 2; ++m) {
        const float* p = a + rho(i, c) * kLd + 32 * m + 8 * lg;
        image_put<kW>(to, lower_frag(i, m), frag_of<kW>(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4)));
      }
  } else {
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int m = j / 2; m < KC; ++m) {
        const float* p = a + (32 * m + 8 * lg) * kLd + rho(j, c);
        f32x4 x, y;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[r] = p[r * kLd];
          y[r] = p[(4 + r) * kLd];
        }
        image_put<kW>(to, upper_frag<KC>(j, m), frag_of<kW>(x, y));
      }
  }
}

// ----------------------------------------------------------------- chain of states
template <typename T>
struct FwdArgs {
  Rows k, q;
  Heads<const T> v;
  Heads<T> o;
  const uint16_t* units;
  const float* s0;
  float *s1, *saved;  // the final state; what the backward needs (delta_saved_floats)
  int image_floats, saved_floats;
};

// Workgroup (x, s): value head x % H of sequence s; wave w takes the columns
// 16 (8 (x / H) + w) .. of v. Heads run fastest, so the workgroups of one head, which
// read the same fragments, meet in one of the eight L2 caches. A chunk's fragments
// come into LDS while the chunk before is worked on; K^T is read there from K's rows.
//
// TEAM: 16 columns and three waves. The first is left with the chain of states; the second forms
// O, a chunk behind, from what that leaves in LDS of S0 and N; the third fetches. (A wave
// that does all of it waits for its loads to be taken: 5.8 us a chunk where the team needs 2.2.)
//
// The state goes from chunk to chunk as itself and as fragments, whose words are made
// while the matrix instructions of the other half of it run.
template <typename T, int DK, bool TEAM>
__global__ __launch_bounds__(512) void delta_fwd_kernel(DeltaSizes z, FwdArgs<T> A) {
  typedef Unit<T, false> Rec;
  constexpr int kIn = DeltaType<T>::kIn, kLogC = DeltaType<T>::kLogC, C = 1 << kLogC;
  constexpr int RT = C / 16, KC = C / 32, DT = DK / 16, KD = DK / 32, kW = kStateWords;
  constexpr int NW = TEAM ? 1 : 8;
  // fragments in LDS: two buffers of K, the inverse and the gates, Q and P; V of each wave (TEAM: two); S0 and N for the team
  constexpr int nRows = RT * KD * kIn, nHead = Rec::oP, nP = Rec::nP, nX = KD * kW + RT;
  constexpr int oQ = nRows + nHead, oP = oQ + nRows, kBuf = oP + nP, oV = 2 * kBuf, oX = oV + (TEAM ? 4 : 2 * NW);
  __shared__ __align__(16) char lds[(oX + (TEAM ? nX : 0)) * 1024];
  const int lane = threadIdx.x & 63, wave_ = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, lg = lane >> 4;
  const int role = TEAM ? wave_ : 0, wave = TEAM ? 0 : wave_;
  const int h = blockIdx.x % z.H, hk = h / (z.H / z.Hk), v0 = ((blockIdx.x / z.H) * NW + wave) * 16, s = blockIdx.y;
  const uint32_t lds0 = lds_address(lds);
  char* x = lds + oX * 1024;
  uint32_t r0, r1, first;
  segment_rows(z.offs, s, static_cast<uint32_t>(z.T), kLogC, r0, r1, first);
  int64_t unit = static_cast<int64_t>(first) * z.H + h;
  int buf = 0;

  const bool whole = whole_columns(A.v, v0, z.dv);
  const auto v_tile = [&](int buf) { return (oV + 2 * (TEAM ? buf : wave)) * 1024; };
  const auto rows_at = [&](uint32_t t0) { return r1 - t0 < static_cast<uint32_t>(C) ? static_cast<int>(r1 - t0) : C; };
  const auto fetch_next = [&](uint32_t t0, int64_t unit, int buf) {
    const uint32_t to = lds0 + buf * kBuf * 1024;
    const uint16_t* rec = A.units + unit * Rec::kElems;
    fetch_rows<RT, KD, kIn, NW>(to, A.k, t0, rows_at(t0) - 1, hk, wave);
    fetch_image<nHead, NW, 4>(to + nRows * 1024, rec, wave);
  };
  const auto fetch_qp = [&](uint32_t t0, int64_t unit, int buf) {
    const uint32_t to = lds0 + buf * kBuf * 1024;
    fetch_rows<RT, KD, kIn, NW, 4>(to + oQ * 1024, A.q, t0, rows_at(t0) - 1, hk, wave);
    fetch_image<nP, NW, 5>(to + oP * 1024, A.units + unit * Rec::kElems + Rec::oP * kFragElems, wave);
  };
  const auto fetch_v = [&](uint32_t t0, int buf) {
    if (whole) fetch_columns<RT>(lds0 + v_tile(buf), A.v, t0, h, v0, rows_at(t0) - 1);
  };

  if (role == 2) {
    if (r0 < r1) {
      fetch_next(r0, unit, 0);
      fetch_v(r0, 0);
      fetch_qp(r0, unit, 0);
    }
    fetch_done();
    for (uint32_t t0 = r0; t0 < r1; t0 += C, unit += z.H, buf ^= 1) {
      __syncthreads();  // this chunk's fragments are there, the last one's have been read, but Q and P
      const bool more = t0 + C < r1;
      if (more) {
        fetch_next(t0 + C, unit + z.H, buf ^ 1);
        fetch_v(t0 + C, buf ^ 1);
      }
      __syncthreads();  // S0 and N are there, the last chunk's Q and P have been read
      if (more) {
        fetch_qp(t0 + C, unit + z.H, buf ^ 1);
        fetch_done_but<nRows + nP>();
      } else {
        fetch_done();
      }
    }
    __syncthreads();
    return;
  }

  if (role == 1) {
    Frag<kW> xs[KD], xu[KC];
    f32x4 nt[RT];
    float eg[RT];
    const auto put_o = [&](uint32_t t0, int64_t unit, int buf) {  // (rows v, columns t)
      const char *q_img = lds + (buf * kBuf + oQ) * 1024, *p_img = lds + (buf * kBuf + oP) * 1024;
      f32x4 o[RT] = {};
#pragma unroll
      for (int ks = 0; ks < KD; ++ks) {
        Frag<kIn> fq[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) fq[i] = row_frag<kIn>(q_img, i * KD + ks);
        mm_tiles<kW, 0, RT, true>(o, fq, xs[ks]);
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) o[i] *= eg[i];
      static_for<KC>([&](auto kt) {
        Frag<kW> fp[RT];
#pragma unroll
        for (int i = 2 * kt.value; i < RT; ++i) fp[i] = lds_frag<kW, kW>(p_img, lower_frag(i, kt.value));
        mm_tiles<kW, 2 * kt.value, RT, true>(o, fp, xu[kt.value]);
      });
      if (A.saved) put_image<RT>(nt, A.saved + unit * A.saved_floats, v0, z.dv, z.dv <= 64 ? 2 : 4);
      store_rows<RT>(o, A.o.row(t0, h), A.o.st, v0, z.dv, rows_at(t0));
    };
    for (uint32_t t0 = r0; t0 < r1; t0 += C, unit += z.H, buf ^= 1) {
      __syncthreads();
      if (t0 > r0) put_o(t0 - C, unit - z.H, buf ^ 1);
      lds_read();
      __syncthreads();  // S0 and N are there
#pragma unroll
      for (int ks = 0; ks < KD; ++ks) xs[ks] = lds_frag<kW, kW>(x, ks);
      const float* gate = reinterpret_cast<const float*>(lds + (buf * kBuf + nRows + Rec::oGate) * 1024);
      char* xn = x + KD * kW * 1024;
#pragma unroll
      for (int kt = 0; kt < KC; ++kt)
        xu[kt] = frag_of<kW>(*lds_tile(xn + 2 * kt * 1024) * gate4(gate, C, kBeta, rho(2 * kt, 4 * lg)),
                               *lds_tile(xn + (2 * kt + 1) * 1024) * gate4(gate, C, kBeta, rho(2 * kt + 1, 4 * lg)));
      if (A.saved)
#pragma unroll
        for (int i = 0; i < RT; ++i) nt[i] = lds_turned(xn + i * 1024);
#pragma unroll
      for (int i = 0; i < RT; ++i) eg[i] = gate[kEG * C + rho(i, c)] * z.scale;
      lds_read();
    }
    __syncthreads();
    if (r0 < r1) put_o(r0 + ((r1 - r0 - 1) >> kLogC << kLogC), unit - z.H, buf ^ 1);
    return;
  }

  // the state's rows rho(i, 4 lg + r), column v0 + c
  const int col = v0 + c, vcol = col < z.dv ? col : z.dv - 1;
  const int64_t size = static_cast<int64_t>(z.dk) * z.dv, of = (static_cast<int64_t>(s) * z.H + h) * size;
  f32x4 S[DT] = {};
  if (A.s0) {
    float y[DT][4];
    load_state<DT>(y, A.s0 + of, z.dk, z.dv, vcol);
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = rho(i, 4 * lg + r) < z.dk ? y[i][r] : 0.0f;
  }
  Frag<kW> f[KD];  // of S
#pragma unroll
  for (int ks = 0; ks < KD; ++ks) f[ks] = frag_of<kW>(S[2 * ks], S[2 * ks + 1]);
  T rv[RT][4];
  const auto next_v = [&](uint32_t t0) {
    if (!whole) {
      load_column<RT>(rv, A.v.row(t0, h), A.v.st, vcol, rows_at(t0) - 1);
    } else if (!TEAM) {
      lds_read();  // (the last one's)
      fetch_v(t0, 0);
    }
  };
  if (r0 < r1) {
    next_v(r0);
    if (!TEAM) {
      fetch_next(r0, unit, 0);
      fetch_qp(r0, unit, 0);
    }
  }
  if (!TEAM) fetch_done();
  for (uint32_t t0 = r0; t0 < r1; t0 += C, unit += z.H, buf ^= 1) {
    __syncthreads();  // this chunk's fragments are there, the last one's have been read
    if (!TEAM && t0 + C < r1) {
      fetch_next(t0 + C, unit + z.H, buf ^ 1);
      fetch_qp(t0 + C, unit + z.H, buf ^ 1);
    }
    const char* img = lds + buf * kBuf * 1024;
    const float* gate = reinterpret_cast<const float*>(img + (nRows + Rec::oGate) * 1024);
    f32x4 R[RT];
    if (whole) {
      take_columns<RT>(R, lds + v_tile(buf), static_cast<const T*>(nullptr));
    } else {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) R[i][r] = to_f32(rv[i][r]);
    }
    if (A.saved && v0 < z.dv) {
      lds_read();
      store_block<DT>(S, A.saved + unit * A.saved_floats + A.image_floats + v0 * z.dk, z.dk, TEAM ? x + KD * kW * 1024 : lds + v_tile(0));
    }

    // K S0 (rows t, columns v) and its transposed Q S0 (rows v, columns t)
    f32x4 ks0[RT] = {}, o[RT] = {};
#pragma unroll
    for (int ks = 0; ks < KD; ++ks) {
      Frag<kIn> fk[RT], fq[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) fk[i] = row_frag<kIn>(img, i * KD + ks);
      if (TEAM) {
        lds_put<kW>(x, ks, f[ks]);
      } else {
#pragma unroll
        for (int i = 0; i < RT; ++i) fq[i] = row_frag<kIn>(img + oQ * 1024, i * KD + ks);
      }
      mm_tiles<kW, 0, RT>(ks0, fk, f[ks]);
      if (!TEAM) mm_tiles<kW, 0, RT, true>(o, fq, f[ks]);
    }
    if (!TEAM)
#pragma unroll
      for (int i = 0; i < RT; ++i) o[i] *= gate[kEG * C + rho(i, c)] * z.scale;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const f32x4 eg = gate4(gate, C, kEG, rho(i, 4 * lg));
#pragma unroll
      for (int r = 0; r < 4; ++r) R[i][r] = __builtin_fmaf(-eg[r], ks0[i][r], R[i][r]);
    }
    if (TEAM && t0 + C < r1) next_v(t0 + C);
    // N
    f32x4 U[RT] = {};
    static_for<KC>([&](auto kt) {
      const Frag<kW> fr = frag_of<kW>(R[2 * kt.value], R[2 * kt.value + 1]);
      Frag<kW> fi[RT];
#pragma unroll
      for (int i = 2 * kt.value; i < RT; ++i) fi[i] = lds_frag<kW, kW>(img + nRows * 1024, lower_frag(i, kt.value));
      mm_tiles<kW, 2 * kt.value, RT>(U, fi, fr);
    });
    if (!TEAM) {
      if (A.saved) {
        f32x4 nt[RT];  // with rows v and columns t
        lds_read();
        turn_tiles<RT>(nt, U, lds + v_tile(0));
        put_image<RT>(nt, A.saved + unit * A.saved_floats, v0, z.dv, z.dv <= 64 ? 2 : 4);
      }
      if (t0 + C < r1) next_v(t0 + C);
    }
    if (TEAM) {
#pragma unroll
      for (int i = 0; i < RT; ++i) *lds_tile(x + (KD * kW + i) * 1024) = U[i];
    } else {
      static_for<KC>([&](auto kt) {
        constexpr int k = 2 * kt.value;
        const Frag<kW> fu = frag_of<kW>(U[k] * gate4(gate, C, kBeta, rho(k, 4 * lg)), U[k + 1] * gate4(gate, C, kBeta, rho(k + 1, 4 * lg)));
        Frag<kW> fp[RT];
#pragma unroll
        for (int i = k; i < RT; ++i) fp[i] = lds_frag<kW, kW>(img + oP * 1024, lower_frag(i, kt.value));
        mm_tiles<kW, k, RT, true>(o, fp, fu);
      });
      store_rows<RT>(o, A.o.row(t0, h), A.o.st, v0, z.dv, rows_at(t0));
    }
    const float el = gate[kEnd * C];
#pragma unroll
    for (int i = 0; i < RT; ++i) U[i] *= gate4(gate, C, kRestBeta, rho(i, 4 * lg));
    if (TEAM) __syncthreads();  // S0 and N are there
    Frag<kW> fu[KC];
#pragma unroll
    for (int kt = 0; kt < KC; ++kt) fu[kt] = frag_of<kW>(U[2 * kt], U[2 * kt + 1]);
    next_state<kIn, KC>(S, f, img, fu, el);
    if (!TEAM) fetch_done();
  }
  if (TEAM) __syncthreads();
  if (A.s1) store_state<DT>(S, A.s1 + of, z.dk, z.dv, col);
}

// Whether the kernels can read a tensor's rows as they are.
bool as_it_is(const void* p, int64_t st, int64_t sh, int64_t dim) {
  return dim == delta_pad(dim) && aligned(p, 16) && st % 8 == 0 && sh % 8 == 0 && st < (1 << 24);
}

// The rows of a tensor, from a copy that joins `all` where need be.
template <typename T>
Rows rows_of(Copies<T>& all, int dtype, const void* x, int64_t x_st, int64_t x_sh, int heads, int dim, uint16_t* copy) {
  if (sizeof(T) == 2 && as_it_is(x, x_st, x_sh, dim)) return {static_cast<const uint16_t*>(x), x_st, x_sh, 0};
  const int pad = delta_pad(dim), words = delta_words(dtype), i = all.n++;
  all.x[i] = {static_cast<const T*>(x), x_st, x_sh};
  all.rows[i] = copy;
  all.heads[i] = heads;
  all.dim[i] = dim;
  all.pad[i] = pad;
  return {copy, static_cast<int64_t>(heads) * words * pad, static_cast<int64_t>(words) * pad, pad};
}

template <typename T, int DK>
void launch_prep(const DeltaSizes& z, bool bwd, const Rows& k, const Rows& q, const float* g, int64_t g_ld, const void* beta,
                 int64_t beta_ld, uint16_t* out, int64_t units, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>(ceil_div(units, kPrepWaves)));
  if (bwd)
    hipLaunchKernelGGL((delta_prep_kernel<T, DK, true>), grid, dim3(64 * kPrepWaves), 0, st, z, k, q, g, g_ld,
                       static_cast<const T*>(beta), beta_ld, out, units);
  else
    hipLaunchKernelGGL((delta_prep_kernel<T, DK, false>), grid, dim3(64 * kPrepWaves), 0, st, z, k, q, g, g_ld,
                       static_cast<const T*>(beta), beta_ld, out, units);
}

template <typename T>
DeltaPrepared prepare(const DeltaSizes& z, int dtype, bool bwd, const void* q, int64_t q_st, int64_t q_sh, const void* k,
                      int64_t k_st, int64_t k_sh, const void* d_o, int64_t do_st, int64_t do_sh, const float* g, int64_t g_ld,
                      const void* beta, int64_t beta_ld, char* ws, const DeltaLayout& l, hipStream_t st) {
  const auto at = [&](size_t o) { return reinterpret_cast<uint16_t*>(ws + o); };
  DeltaPrepared r{};
  Copies<T> all{};
  r.k = rows_of<T>(all, dtype, k, k_st, k_sh, z.Hk, z.dk, at(l.k_rows));
  r.q = rows_of<T>(all, dtype, q, q_st, q_sh, z.Hk, z.dk, at(l.q_rows));
  if (bwd) r.d_o = rows_of<T>(all, dtype, d_o, do_st, do_sh, z.H, z.dv, at(l.o_rows));
  if (all.n) {
    const dim3 grid(static_cast<uint32_t>(delta_tiles(z.T, z.S, dtype)), static_cast<uint32_t>(bwd ? z.H : z.Hk), static_cast<uint32_t>(all.n));
    hipLaunchKernelGGL(delta_copy_kernel<T>, grid, dim3(256), 0, st, z, all);
  }
  const int64_t units = delta_tiles(z.T, z.S, dtype) * z.H;
  if (z.dk <= 64) launch_prep<T, 64>(z, bwd, r.k, r.q, g, g_ld, beta, beta_ld, at(l.units), units, st);
  else launch_prep<T, 128>(z, bwd, r.k, r.q, g, g_ld, beta, beta_ld, at(l.units), units, st);
  return r;
}

template <typename T, int DK>
void launch_fwd(const DeltaSizes& z, const FwdArgs<T>& A, hipStream_t st) {
  const bool teams = delta_teams(z);
  const int64_t columns = A.saved ? delta_pad(z.dv) : z.dv;  // (the images' padding is written too)
  const dim3 grid(static_cast<uint32_t>(z.H * ceil_div(columns, teams ? 16 : 128)), static_cast<uint32_t>(z.S));
  if (teams) hipLaunchKernelGGL((delta_fwd_kernel<T, DK, true>), grid, dim3(192), 0, st, z, A);
  else hipLaunchKernelGGL((delta_fwd_kernel<T, DK, false>), grid, dim3(512), 0, st, z, A);
}

}  // namespace

DeltaLayout delta_layout(const DeltaSizes& z, int dtype, bool bwd) {
  const int64_t tiles = delta_tiles(z.T, z.S, dtype), units = tiles * z.H;
  const int64_t words = delta_words(dtype), dk = delta_pad(z.dk), dv = delta_pad(z.dv);
  const int64_t unit = dtype == DET_BF16 ? (bwd ? Unit<uint16_t, true>::kElems : Unit<uint16_t, false>::kElems)
                                         : (bwd ? Unit<float, true>::kElems : Unit<float, false>::kElems);
  DeltaLayout l{};
  size_t at = DET_WS_HEADER_BYTES;
  const auto take = [&](int64_t bytes) {
    const size_t r = at;
    at += align_up(static_cast<size_t>(bytes), 256);
    return r;
  };
  l.units = take(units * unit * 2);
  l.k_rows = take(z.T * z.Hk * words * dk * 2);
  l.q_rows = take(z.T * z.Hk * words * dk * 2);
  l.o_rows = take(bwd ? z.T * z.H * words * dv * 2 : 0);
  l.ds = take(bwd ? units * delta_block_floats(z.dk, z.dv) * 4 : 0);
  l.dy = take(bwd ? units * delta_image_floats(z.dv, dtype) * 4 : 0);
  l.all = at;
  return l;
}

DeltaPrepared delta_prepare(const DeltaSizes& z, int dtype, bool bwd, const void* q, int64_t q_st, int64_t q_sh, const void* k,
                            int64_t k_st, int64_t k_sh, const void* d_o, int64_t do_st, int64_t do_sh, const float* g,
                            int64_t g_ld, const void* beta, int64_t beta_ld, char* ws, const DeltaLayout& l, hipStream_t st) {
  if (dtype == DET_BF16)
    return prepare<uint16_t>(z, dtype, bwd, q, q_st, q_sh, k, k_st, k_sh, d_o, do_st, do_sh, g, g_ld, beta, beta_ld, ws, l, st);
  return prepare<float>(z, dtype, bwd, q, q_st, q_sh, k, k_st, k_sh, d_o, do_st, do_sh, g, g_ld, beta, beta_ld, ws, l, st);
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

extern "C" int det_delta_rule_states_size(int64_t T, int64_t S, int64_t dk, int64_t dv, int dtype, int64_t* chunks,
                                          int64_t* floats) {
  if (!chunks || !floats) return set_error(DET_ERR_INVALID_ARG, "delta_rule: chunks or floats is NULL");
  if (int s = delta_check_sizes("delta_rule", dtype, T, S, 1, 1, dk, dv)) return s;
  *chunks = delta_tiles(T, S, dtype);
  *floats = delta_saved_floats(dk, dv, dtype);
  return ok();
}

extern "C" int det_delta_rule_workspace_size(int64_t T, int64_t S, int64_t Hk, int64_t H, int64_t dk, int64_t dv, int dtype,
                                             size_t* bytes) {
  if (!bytes) return set_error(DET_ERR_INVALID_ARG, "delta_rule: bytes is NULL");
  if (int s = delta_check_sizes("delta_rule", dtype, T, S, Hk, H, dk, dv)) return s;
  const DeltaSizes z{T, (int)S, (int)Hk, (int)H, (int)dk, (int)dv, nullptr, 0.0f};
  *bytes = T == 0 ? 0 : delta_layout(z, dtype, false).all;
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
  const DeltaLayout l = delta_layout(z, dtype, false);
  const size_t need = T ? l.all : 0;
  if (int s = check_workspace(ws, ws_bytes, need)) return s;
  const size_t state = static_cast<size_t>(H * dk * dv) * 4;
  const Buf outs[] = {bo,
                      {"final_state", range1d(final_state, S * state)},
                      {"states", range1d(states, delta_tiles(T, S, dtype) * H * delta_saved_floats(dk, dv, dtype) * 4), 16},
                      {"the workspace", range1d(need ? ws : nullptr, ws_bytes)}};
  const Buf ins[] = {bq, bk, bv, buf_rows("g", g, T, H, T > 1 ? g_ld : H, 4),
                     buf_rows("beta", beta, T, H, T > 1 ? beta_ld : H, es),
                     {"offs", range1d(offs, (S + 1) * 4)},
                     {"initial_state", range1d(initial_state, S * state)}};
  if (int s = check_buffers(what, outs, 4, ins, 7)) return s;
  const hipStream_t st = as_stream(stream);
  char* base = static_cast<char*>(ws);  // (no tokens: nothing there is read)
  DeltaPrepared r{};
  if (T)
    r = delta_prepare(z, dtype, false, q, q_st, q_sh, k, k_st, k_sh, nullptr, 0, 0, g, g_ld, beta, beta_ld, base, l, st);
#define DET_DELTA_FWD(E)                                                                                            \
  {                                                                                                                 \
    const FwdArgs<E> A{r.k, r.q, {static_cast<const E*>(v), v_st, v_sh}, {static_cast<E*>(o), o_st, o_sh},          \
                       reinterpret_cast<const uint16_t*>(base + l.units),                                           \
                       initial_state, final_state, states, (int)delta_image_floats(dv, dtype),                      \
                       (int)delta_saved_floats(dk, dv, dtype)};                                                       \
    if (dk <= 64) launch_fwd<E, 64>(z, A, st);                                                                      \
    else launch_fwd<E, 128>(z, A, st);                                                                              \
  }
  if (dtype == DET_BF16) DET_DELTA_FWD(uint16_t)
  else DET_DELTA_FWD(float)
#undef DET_DELTA_FWD
  return check_launch("det_delta_rule");
}
