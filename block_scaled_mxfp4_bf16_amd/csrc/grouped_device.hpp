// Ragged groups of rows, shared by the kernels of the grouped product.
//
// Expert e owns the output rows offsets[e] .. offsets[e + 1] - 1.  Its
// quantized rows lie in the workspace in "quads" of 64 rows, the last one
// partly filled, the quads of one expert consecutive and the experts in
// order, each quad in the operand layout of the large-M product:
//   codes   16-row tile t, K step ks: 1 KiB at (t * KS + ks) * 1024, operand
//           lane L's 16 bytes at 16 * L (row 16 t + L % 16, K chunk L / 16);
//   scales  quad q, K step ks: 256 bytes at (q * KS + ks) * 256.  For the
//           16-row instruction dword L holds operand lane L's scale bytes of
//           the quad's four tiles; for the 32-row one (`pairs`) byte 2 t + h of
//           dword L is that of row 32 t + L % 32, K chunk 2 h + L / 32.
// Tiles without a row are never written nor read.
//
// The product walks over "units", runs of 16, 64 or 128 rows of one expert,
// that the first launch lists in the workspace: the group sizes are known on
// the device only, and one 16-byte entry is cheaper for a workgroup to read
// than E offsets to scan.
#pragma once

#include "experts_bounds.hpp"
#include "experts_device.hpp"
#include "experts_internal.hpp"

namespace mxfp4 {

// plan[0].x is the number of units, plan[1 + u] unit u.  Entries are read
// through the scalar cache: the index is the same in every lane, and the reads
// do not queue behind the operand loads.  Both are held to this call's sizes.
typedef int i32x4 __attribute__((ext_vector_type(4)));
template <int UNIT_ROWS>
__device__ __forceinline__ Unit plan_entry(const GroupedArgs &a, int i) {
  const i32x4 v = ((const __attribute__((address_space(4))) i32x4 *)a.plan)[i];
  int w[4] = {v.x, v.y, v.z, v.w};
  // what is checked is what is used: no second read in its place
  asm("" : "+s"(w[0]), "+s"(w[1]), "+s"(w[2]), "+s"(w[3]));
  return unit_of(w[0], w[1], w[2], w[3], a.R, a.E, 4 * a.quads, UNIT_ROWS);
}

__device__ __forceinline__ int unit_count(const GroupedArgs &a) {
  int n = *(const __attribute__((address_space(4))) int *)a.plan;
  asm("" : "+s"(n));
  return within(n, 0, a.max_units);
}

// Rows of expert e, clamped to [0, R): whatever the offsets hold, no group
// reaches outside the output.
__device__ __forceinline__ void group_range(const GroupedArgs &a, int e, int &lo, int &hi) {
  const int p = a.offsets[e], q = a.offsets[e + 1];
  lo = p < 0 ? 0 : (p > a.R ? a.R : p);
  hi = q < lo ? lo : (q > a.R ? a.R : q);
}

// Inclusive sums over the lanes of a wave: shifts by 1, 2, 4 and 8 within the
// rows of 16 lanes, then the last lane of row 0 (2) added to row 1 (3) and that
// of lane 31 to the upper half.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// One wave's view of the groups: each lane holds the sums over its share of
// the experts, a scan over the lanes says where the share starts.
struct GroupScan {
  int first_e, last_e;         // this lane's experts
  int units_before, quads_before;
  int units, quads;            // of all experts

  __device__ __forceinline__ GroupScan(const GroupedArgs &a, int lane) {
    const int per = (a.E + 63) >> 6;
    first_e = lane * per < a.E ? lane * per : a.E;
    last_e = first_e + per < a.E ? first_e + per : a.E;
    int u = 0, q = 0;
    for (int e = first_e; e < last_e; ++e) {
      int lo, hi;
      group_range(a, e, lo, hi);
      u += (hi - lo + a.unit_rows - 1) >> a.unit_shift;
      q += (hi - lo + 63) >> 6;
    }
    const int ui = wave_scan(u), qi = wave_scan(q);
    units_before = ui - u;
    quads_before = qi - q;
    units = __builtin_amdgcn_readlane(ui, 63);
    quads = __builtin_amdgcn_readlane(qi, 63);
  }

  // The quad with the given index (below `quads`, the same in every lane).
  __device__ __forceinline__ Unit quad(const GroupedArgs &a, int index) const {
    int expert = -1, row = 0, rows = 0;
    int q = quads_before;
    for (int e = first_e; e < last_e; ++e) {
      int lo, hi;
      group_range(a, e, lo, hi);
      const int n = (hi - lo + 63) >> 6;
      if (index >= q && index < q + n) {
        expert = e;
        row = lo + (index - q) * 64;
        rows = hi - row;
      }
      q += n;
    }
    const int src = __builtin_ctzll(__ballot(expert >= 0) | (1ull << 63));
    return Unit{__builtin_amdgcn_readlane(expert, src), __builtin_amdgcn_readlane(row, src),
                __builtin_amdgcn_readlane(rows, src), index * 4, 0};
  }

  // Lists the units.  Offsets that do not rise can describe more units and
  // quads than R rows can take; what lies past the workspace is left out.
  __device__ __forceinline__ void list(const GroupedArgs &a, int lane) const {
    int u = units_before, q = quads_before;
    for (int e = first_e; e < last_e; ++e) {
      int lo, hi;
      group_range(a, e, lo, hi);
      const int last_quad = q + ((hi - lo + 63) >> 6);
      int first = e;  // the entry's first word
      for (int row = lo, tile = 4 * q; row < hi; row += a.unit_rows, tile += a.unit_rows >> 4, ++u) {
        const bool fits = last_quad <= a.quads;
        if (u < a.max_units) a.plan[1 + u] = int4{fits ? first : -1, row, fits ? hi - row : 0, tile};
        first += kMaxExperts;
      }
      q = last_quad;
    }
    if (lane == 0) a.plan[0] = int4{units < a.max_units ? units : a.max_units, 0, 0, 0};
  }
};

__device__ __forceinline__ v4f mfma_fp4(const u32x4 &a, const u32x4 &b, const v4f &c, uint32_t sa, uint32_t sb) {
  const v8i av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

}  // namespace mxfp4
