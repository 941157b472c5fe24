// Ragged groups of rows, shared by the kernels of the grouped product.
//
// Expert e owns the output rows offsets[e] .. offsets[e + 1] - 1.  Its
// quantized rows lie in the workspace in "quads" of 64 rows, the last one
// partly filled, the quads of one expert consecutive and the experts in
// order, each quad in the operand layout of the large-M product:
//   codes   16-row tile t, K step ks: 1 KiB at (t * KS + ks) * 1024, operand
//           lane L's 16 bytes at 16 * L (row 16 t + L % 16, K chunk L / 16);
//   scales  quad q, K step ks: 256 bytes at (q * KS + ks) * 256, dword L the
//           scale bytes of operand lane L of the quad's four tiles.
// Tiles without a row are never written nor read.
#pragma once

#include "experts_device.hpp"

namespace mxfp4 {

// A run of rows of one group.
struct Unit {
  int expert;  // -1: no such unit
  int row;     // first output row
  int rows;    // output rows from `row` to the end of the group
  int tile;    // its first 16-row tile in the workspace
};

__device__ __forceinline__ void group_range(const int32_t *offsets, int e, int R, int &lo, int &hi) {
  const int a = offsets[e], b = offsets[e + 1];
  lo = a < 0 ? 0 : (a > R ? R : a);
  hi = b < lo ? lo : (b > R ? R : b);
}

__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Finds units of UR rows (a multiple of 16): every lane of a wave adds up the
// units and quads of its share of the experts, and a scan over the lanes says
// where each share starts.  All offsets are clamped to [0, R], so no group
// reaches outside the output whatever they hold.
template <int UR>
struct UnitFinder {
  int lane, per, first_e, last_e;
  int units_before, quads_before, total;
  const int32_t *offsets;
  int R;

  __device__ __forceinline__ UnitFinder(const int32_t *off, int E, int R_, int lane_) : lane(lane_), offsets(off), R(R_) {
    per = (E + 63) >> 6;
    first_e = lane * per < E ? lane * per : E;
    last_e = first_e + per < E ? first_e + per : E;
    int u = 0, q = 0;
    for (int e = first_e; e < last_e; ++e) {
      int lo, hi;
      group_range(offsets, e, R, lo, hi);
      u += (hi - lo + UR - 1) / UR;
      q += (hi - lo + 63) >> 6;
    }
    const int ui = wave_scan(u, lane), qi = wave_scan(q, lane);
    units_before = ui - u;
    quads_before = qi - q;
    total = __builtin_amdgcn_readlane(ui, 63);
  }

  // index < total, the same in every lane
  __device__ __forceinline__ Unit find(int index) const {
    int e_found = -1, row = 0, rows = 0, tile = 0;
    int u = units_before, q = quads_before;
    for (int e = first_e; e < last_e; ++e) {
      int lo, hi;
      group_range(offsets, e, R, lo, hi);
      const int n = (hi - lo + UR - 1) / UR;
      if (index >= u && index < u + n) {
        const int skip = (index - u) * UR;
        e_found = e;
        row = lo + skip;
        rows = hi - row;
        tile = q * 4 + (skip >> 4);
      }
      u += n;
      q += (hi - lo + 63) >> 6;
    }
    const int src = __builtin_ctzll(__ballot(e_found >= 0) | (1ull << 63));
    Unit r;
    r.expert = __builtin_amdgcn_readlane(e_found, src);
    r.row = __builtin_amdgcn_readlane(row, src);
    r.rows = __builtin_amdgcn_readlane(rows, src);
    r.tile = __builtin_amdgcn_readlane(tile, src);
    return r;
  }
};

}  // namespace mxfp4
