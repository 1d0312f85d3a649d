// Tiles of segments whose bounds lie in a device offset array: used by every
// kernel whose workgroups own a block of rows of one segment (an expert's rows,
// a sequence's tokens) while the host knows only the worst-case tile count.
#pragma once

#include "common.hpp"

namespace detgrad {

// Inclusive scans over the 64 lanes on DPP (row shifts by 1, 2, 4, 8, then
// the last lane of row 0 into rows 1 and 3 and of row 1 into rows 2 and 3);
// lanes without a source read 0, the identity of both (the values are >= 0).
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t dpp_src(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROW_MASK, 0xF, false));
}
__device__ __forceinline__ uint32_t scan_add(uint32_t v) {
  v += dpp_src<0x111, 0xF>(v); v += dpp_src<0x112, 0xF>(v); v += dpp_src<0x114, 0xF>(v);
  v += dpp_src<0x118, 0xF>(v); v += dpp_src<0x142, 0xA>(v); v += dpp_src<0x143, 0xC>(v);
  return v;
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t scan_max(uint32_t v) {
  v = umax(v, dpp_src<0x111, 0xF>(v)); v = umax(v, dpp_src<0x112, 0xF>(v)); v = umax(v, dpp_src<0x114, 0xF>(v));
  v = umax(v, dpp_src<0x118, 0xF>(v)); v = umax(v, dpp_src<0x142, 0xA>(v)); v = umax(v, dpp_src<0x143, 0xC>(v));
  return v;
}
// the value of the lane below, `fill` in lane 0 (DPP wave_shr:1 with the fill
// as the old value; computed with every lane active, never under a branch)
__device__ __forceinline__ uint32_t from_lane_below(uint32_t v, uint32_t fill) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(static_cast<int>(fill), static_cast<int>(v), 0x138, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int j) {
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), j));
}
__device__ __forceinline__ uint32_t clamp_off(int32_t o, uint32_t M) {
  const uint32_t v = o < 0 ? 0u : static_cast<uint32_t>(o);
  return v < M ? v : M;
}

// Segment tile table, computed by every workgroup from the device offsets:
// b_e = min(M, max(0, offs[0..e])) (clamped monotone), tiles_e =
// ceil((b_{e+1} - b_e) / block_m), tile_start_e = sum of tiles before e.
// Returns the segment of global tile t (false past the last tile), the tile's
// rows [r0, r1) and the segment's rows [s0, s1). BATCH groups of 64 offsets are
// fetched together (one group at a time suffices for a few experts).
template <int BATCH>
__device__ __forceinline__ bool segment_tile(const int32_t* __restrict__ offs, int E, uint32_t M, int log_bm,
                                             uint32_t t, int& e_out, uint32_t& r0, uint32_t& r1, uint32_t& s0,
                                             uint32_t& s1) {
  const int lane = threadIdx.x & 63;
  const uint32_t bm = 1u << log_bm;
  uint32_t run_b = clamp_off(offs[0], M);  // b of the first segment of the chunk
  uint32_t run_t = 0;                      // tiles before the chunk
  for (int e1 = 0; e1 < E; e1 += 64 * BATCH) {
    uint32_t next[BATCH];  // the clamped offsets e + 1 (lanes past E repeat offs[E])
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (BATCH > 1 && k > 0 && e1 + 64 * k >= E) break;
      const int e = e1 + 64 * k + lane;
      next[k] = clamp_off(offs[e < E ? e + 1 : E], M);
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (BATCH > 1 && e1 + 64 * k >= E) break;
      const int e0 = e1 + 64 * k, e = e0 + lane;
      const uint32_t b1 = umax(scan_max(next[k]), run_b);  // b_{e+1}: running max of the offsets
      const uint32_t b0 = from_lane_below(b1, run_b);
      const uint32_t nt = (e < E && b1 > b0) ? (b1 - b0 + bm - 1) >> log_bm : 0u;
      const uint32_t incl = scan_add(nt);
      const uint32_t first = run_t + incl - nt;
      const uint64_t hit = __ballot(e < E && t >= first && t < first + nt);
      if (hit) {
        const int j = __builtin_ctzll(hit);
        e_out = e0 + j;
        s0 = lane_value(b0, j);
        s1 = lane_value(b1, j);
        r0 = s0 + ((t - lane_value(first, j)) << log_bm);
        r1 = s1 - r0 > bm ? r0 + bm : s1;
        return true;
      }
      run_t += lane_value(incl, 63);
      run_b = lane_value(b1, 63);
    }
  }
  return false;
}

// segment_tile without the segment's bounds.
__device__ inline bool tile_of(const int32_t* __restrict__ offs, int E, uint32_t M, int log_bm, uint32_t t, int& e_out,
                               uint32_t& r0, uint32_t& r1) {
  uint32_t s0, s1;
  return segment_tile<1>(offs, E, M, log_bm, t, e_out, r0, r1, s0, s1);
}

// The tile table [E+1] for a fold kernel: table[e] = tiles of the segments before
// e, table[E] = all tiles. Run by one wave (every lane active).
__device__ __forceinline__ void write_tile_table(const int32_t* __restrict__ offs, int E, uint32_t M, int log_bm,
                                                 int32_t* __restrict__ table) {
  const int lane = threadIdx.x & 63;
  const uint32_t bm = 1u << log_bm;
  uint32_t run_b = 0, run_t = 0;
  for (int e0 = 0; e0 <= E; e0 += 64) {
    const int ee = e0 + lane;
    const uint32_t b = umax(scan_max(clamp_off(ee <= E ? offs[ee] : 0, M)), run_b);    // b_ee
    const uint32_t bp = from_lane_below(b, e0 == 0 ? b : run_b);                      // b_{ee-1}
    const uint32_t nt = (ee >= 1 && ee <= E && b > bp) ? (b - bp + bm - 1) >> log_bm : 0u;  // tiles of segment ee-1
    const uint32_t incl = scan_add(nt);
    if (ee <= E) table[ee] = static_cast<int32_t>(run_t + incl);  // tiles of segments before ee
    run_t += lane_value(incl, 63);
    run_b = lane_value(b, 63);
  }
}

}  // namespace detgrad
