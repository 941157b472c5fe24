// The grouped product for groups of many rows (template; instantiated by
// grouped_kernels.hip): 128 rows x 256 weight rows per workgroup, two
// workgroups on a CU.
//
// The four waves share the 128 rows and split the columns, 64 each, so
//   - a block of weights is needed by one wave only and goes from memory to
//     its registers, three K steps ahead;
//   - the rows go through LDS, one 8 KiB slot per K step written directly by
//     the memory system, four slots in a ring; LDS then serves 40 KiB a step
//     and workgroup, where staging the weights as well would take 72 and make
//     LDS the bound;
//   - the weights are the first operand of the matrix instruction: a lane then
//     holds four neighbouring columns of one row and stores 8 bytes.
// Workgroups stay and walk over tiles; the loads run on into the next tile
// while the last steps and the stores of this one are under way.
//
// What a CU takes in bounds it: 48 KiB a K step for its two tiles in 0.93 us, of
// which the matrix units work 0.43.  32768 rows of 64 experts, 4096 x 2048 gated:
// 173 us, 3.2 PFLOP/s (a call among others less its packing; under the profiler,
// between whose launches the clocks move, medians of 183 to 207 and 160 at least);
// 2048 x 2048: 96 us, 2.9 PFLOP/s (medians 100 to 105, least 92).
#pragma once

#include <type_traits>

#include "grouped_device.hpp"

namespace mxfp4 {

// Barrier of LDS written by the memory system: the caller has waited for its
// own loads; nothing may move across.
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// As mfma_fp4_sel2 for 32 x 32 outputs and 64 of K.
typedef float v16f __attribute__((ext_vector_type(16)));
template <int IA>
__device__ __forceinline__ v16f mfma32_fp4_at(const v8i &a, const v8i &b, const v16f &c, uint32_t sa, uint32_t sb, int ib) {
  switch (ib) {
    case 0: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, IA, (int)sa, 0, (int)sb);
    case 1: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, IA, (int)sa, 1, (int)sb);
    case 2: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, IA, (int)sa, 2, (int)sb);
    default: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, IA, (int)sa, 3, (int)sb);
  }
}
__device__ __forceinline__ v16f mfma32_fp4_sel2(const u32x4 &a, const u32x4 &b, const v16f &c, uint32_t sa, int ia,
                                                uint32_t sb, int ib) {
  const v8i av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return ia ? mfma32_fp4_at<2>(av, bv, c, sa, sb, ib) : mfma32_fp4_at<0>(av, bv, c, sa, sb, ib);
}

// The units of an expert are taken in blocks of up to kBlockUnits, the unit
// fastest within a block, so that the workgroups of an XCD that read the same
// weights do it at the same time and the second reader finds them in L2.
// Column tiles fastest instead made 32768 rows of 64 experts, 4096 x 2048 gated,
// read 865 MB through L2 where this reads 400 (199 against 193 us a call).
constexpr int kBlockUnits = 8;

template <bool GATED>
__global__ __launch_bounds__(256, 2) void grouped_tile_kernel(const GroupedArgs a, int n_tiles, int wide_stores) {
  constexpr int MT = 4;       // 32-row tiles of a unit
  constexpr int UT = 2 * MT;  // its 16-row blocks
  constexpr int BN = GATED ? 128 : 256;  // output columns of a tile
  constexpr int STORES = MT * (GATED ? 2 : 4);  // of a wave and tile, 16 bytes a lane
  constexpr int CHUNKS = GATED ? 4 : 8;  // of 8 columns, of a wave
  __shared__ __attribute__((aligned(16))) uint8_t slot0[UT * 1024];
  __shared__ __attribute__((aligned(16))) uint8_t slot1[UT * 1024];
  __shared__ __attribute__((aligned(16))) uint8_t slot2[UT * 1024];
  __shared__ __attribute__((aligned(16))) uint8_t slot3[UT * 1024];
  __shared__ __attribute__((aligned(16))) uint8_t turned[4 * 32 * CHUNKS * 16];
  const auto slot = [&](int s) -> uint8_t * { return s == 0 ? slot0 : (s == 1 ? slot1 : (s == 2 ? slot2 : slot3)); };

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane * 16, l4 = lane * 4;
  // The 32x32x64 instruction takes row lane % 32 and K chunk lane / 32 of one
  // half of a step; a 32-row tile is two blocks of 16 rows x 4 chunks.
  const int r1 = (lane >> 4) & 1, hi = lane >> 5;
  const int in_block = (lane & 15) * 16 + hi * 256;  // + 512 for the second half
  const int N = a.N, K = a.K;
  const int KS = (K + 127) >> 7;
  const int steps = (KS + 3) & ~3;  // steps past K load and add nothing
  const int gp = ((K >> 5) + 7) & ~7;
  const int b_bytes = (N >> 4) * K * 8;
  const int s_bytes = ((N + 255) >> 8) * 8 * gp * 32;
  const int out_cols = GATED ? N >> 1 : N;

  // Workgroup b runs on XCD b % 8.  Each XCD takes a contiguous range of the
  // items (unit, n tile), so that an expert's weights and rows stay in one L2.
  const int units = unit_count(a);
  const int items = units * n_tiles;
  const int xcd = blockIdx.x & 7;
  const int stride = gridDim.x >> 3;
  const int end = (int)((int64_t)items * (xcd + 1) >> 3);
  int next_item = (int)((int64_t)items * xcd >> 3) + (blockIdx.x >> 3);
  if (next_item >= end) return;

  // What the loads of a tile need.  Offsets that all lanes share go into the
  // instructions' scalar offset, which the range check includes: an offset at
  // the end of a buffer or past it reads zeros, as does a buffer of size 0 (no
  // tile left, a tile of no rows, a step past K).
  const uint8_t *a_base, *as_base, *b_base, *s_base;
  int a_size, as_size, b_size, s_size;
  int b_off[2], s_off[2];  // of the wave's two pairs of 16-row groups, and of their scales
  Unit unit;               // of the tile that the loads are in
  int col0;                // its first output column of this wave
  bool none;

  auto enter = [&]() {
    none = next_item >= end;
    const int u = none ? 0 : next_item / n_tiles;
    int n_tile = 0;
    unit = plan_entry<16 * UT>(a, 1 + u);
    if (!none && unit.expert >= 0) {
      const TilePlace at = tile_place(next_item, n_tiles, units, u, unit.index, unit.rows, 16 * UT, kBlockUnits);
      n_tile = at.column;
      unit = plan_entry<16 * UT>(a, 1 + at.unit);
    }
    next_item += stride;
    const int tiles = none || unit.expert < 0 ? 0 : (unit.rows < 16 * UT ? (unit.rows + 15) >> 4 : UT);
    const int64_t expert = unit.expert < 0 ? 0 : unit.expert;
    a_size = tiles * KS * 1024;
    as_size = ((tiles + 3) >> 2) * KS * 256;
    b_size = tiles ? b_bytes : 0;
    s_size = tiles ? s_bytes : 0;
    a_base = a.codes + (int64_t)unit.tile * KS * 1024;
    as_base = a.scales + (int64_t)(unit.tile >> 2) * KS * 256;
    b_base = a.Bw + expert * b_bytes;
    s_base = a.Bs + expert * s_bytes;
    col0 = n_tile * BN + wave * (BN / 4);
    const int g = col0 >> 4;
    const int up = GATED ? N >> 5 : 2;
    const bool ok0 = GATED ? g < (N >> 5) : g < (N >> 4);
    const bool ok1 = GATED ? ok0 : g + 2 < (N >> 4);
    b_off[0] = ok0 ? g * K * 8 : b_bytes;
    b_off[1] = ok1 ? (g + up) * K * 8 : b_bytes;
    s_off[0] = ok0 ? (g >> 1) * gp * 32 : s_bytes;
    s_off[1] = ok1 ? ((g + up) >> 1) * gp * 32 : s_bytes;
  };
  const auto sized = [](const uint8_t *base, int size) {
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, size, kRsrcWord3);
  };

  struct Stage {
    u32x4 b[2][2];    // [32-column tile][half of the step]
    uint32_t as[2];   // of each 64 rows: byte 2 * (32-row tile) + half
    uint32_t bs[2];   // of an even step and the next one, as prepared; unused in odd stages
  };
  Stage st[4];
  const int b_lane = in_block + r1 * K * 8;
  // Part p of the loads of step k0 + s of the loads' tile, into slot and stage
  // s; the eight parts go out between the products of a step, since a wave
  // that issues them in one run waits for the address unit (16 cycles a KiB)
  // and leaves the matrix unit idle.
  auto load_part = [&](int k0, int s, int p) {
    const bool ok = k0 + s < KS;
    if (p == 0) {
      // the weights' scales of this step and the one before, whose stage is
      // loaded but not yet in use; at an odd step the old ones are done with
      const bool any = k0 + s - 1 < KS;
      if (s & 1)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          st[s - 1].bs[q] = __builtin_amdgcn_raw_buffer_load_b32(sized(s_base, any ? s_size : 0), l4 + (s >> 1) * 256,
                                                                 s_off[q] + k0 * 128, 0);
    } else if (p < 3) {  // rows: two of their blocks by each wave
      const int t = 2 * wave + p - 1;
      const __amdgpu_buffer_rsrc_t r = sized(a_base, ok ? a_size : 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)(slot(s) + t * 1024), 16, l16,
                                               (t * KS + k0 + s) * 1024, 0, 0);
    } else if (p < 7) {
      const int nt = (p - 3) >> 1, h = (p - 3) & 1;
      st[s].b[nt][h] = __builtin_amdgcn_raw_buffer_load_b128(sized(b_base, ok ? b_size : 0), b_lane + s * 1024 + h * 512,
                                                             b_off[nt] + k0 * 1024, 0);
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        st[s].as[q] = __builtin_amdgcn_raw_buffer_load_b32(sized(as_base, ok ? as_size : 0), l4 + s * 256,
                                                           (q * KS + k0) * 256, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // Rows 32 mt + lane % 32 of the wave, half h of the step in slot s.
  auto row_block = [&](int s, int i) {
    const int mt = i >> 1, h = i & 1;
    return *(const u32x4 *)(slot(s) + 2 * mt * 1024 + h * 512 + r1 * 1024 + in_block);
  };

  v16f acc[MT][2];
  auto clear = [&]() {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[mt][nt][i] = 0.f;
  };
  auto store = [&](const Unit &u, int col, auto wide) {
    const int rows = u.expert < 0 ? 0 : (u.rows < 32 * MT ? u.rows : 32 * MT);
    const int ldc = (int)a.ldc * 2;
    const __amdgpu_buffer_rsrc_t c_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(a.C + (int64_t)u.row * a.ldc), 0, rows ? (rows - 1) * ldc + out_cols * 2 : 0, kRsrcWord3);
    // Element 4 j + r of an accumulator is column 8 j + 4 * (lane / 32) + r of
    // row lane % 32.  A swap of the upper half of the lanes in j = 2 p with the
    // lower half in j = 2 p + 1 leaves each lane eight neighbouring columns, 16
    // bytes.  Stored as they lie, two lanes of a row would write 32 bytes of
    // it; through LDS, 32 rows at a time, a store covers all of the wave's
    // columns of a row (32768 rows of 64 experts, least times: 2048 x 2048 102 us
    // without, 91 with it; 4096 x 2048 gated, half the columns: 169 and 166).
    // The lane number is found anew for each tile, from a zero that the
    // compiler cannot see through: it would keep the offsets of every store
    // through the products otherwise, and has no registers for them.
    uint32_t zero = 0;
    asm volatile("" : "+s"(zero));
    const int me = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero));
    uint8_t *const turn = turned + wave * 32 * CHUNKS * 16;
    const auto place = [&](int row, int chunk) {  // of a chunk of 8 columns; no two rows of a group in the same banks
      return (u32x4 *)(turn + (row * CHUNKS + (chunk ^ ((CHUNKS == 8 ? row : row >> 1) & (CHUNKS - 1)))) * 16);
    };
    const int chunk = me & (CHUNKS - 1), first_row = me / CHUNKS;
    const int at = first_row * ldc + (col + 8 * chunk) * 2;
    const bool col_ok = col + 8 * chunk < out_cols;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int part = 0; part < CHUNKS / 2; ++part) {
        const int nt = part >> 1, p = part & 1;
        uint32_t d[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = 8 * p + 4 * j + r;
            v[r] = GATED ? gated_silu(acc[mt][0][i], acc[mt][1][i]) : acc[mt][nt][i];
          }
          d[j][0] = bf16x2_rne(v[0], v[1]);
          d[j][1] = bf16x2_rne(v[2], v[3]);
        }
        swap32(d[0][0], d[1][0]);
        swap32(d[0][1], d[1][1]);
        *place(me & 31, 2 * part + (me >> 5)) = u32x4{d[0][0], d[0][1], d[1][0], d[1][1]};
        __builtin_amdgcn_sched_barrier(0);  // few values at a time: the registers are full
      }
      wave_lds_fence();
#pragma unroll
      for (int s = 0; s < CHUNKS / 2; ++s) {
        const int row = s * (64 / CHUNKS) + first_row;
        const u32x4 d = *place(row, chunk);
        const int off = off_or_oob(col_ok && 32 * mt + row < rows, at + (32 * mt + s * (64 / CHUNKS)) * ldc);
        if constexpr (decltype(wide)::value) {
          __builtin_amdgcn_raw_buffer_store_b128(d, c_rsrc, off, 0, 0);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)d[i], c_rsrc, off, 4 * i, 0);
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(d[i] >> 16), c_rsrc, off, 4 * i + 2, 0);
          }
        }
      }
      wave_lds_fence();  // before the next rows
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Loads go out three steps ahead, in step order: the weights' scales (2 loads,
  // for odd steps), the rows (2), the weights and the rows' scales (6).  At the
  // start of step i at least the 14 newest (16 if i is odd) came after
  // rows(i + 1).  The scheduling barriers keep the compiler from mixing them:
  // the load counter retires in issue order.
  u32x4 x[4];
  uint32_t wscale[2][2];
  enter();
#pragma unroll
  for (int s = 0; s < 3; ++s)
#pragma unroll
    for (int p = 0; p < 8; ++p) load_part(0, s, p);
  wait_vmcnt<24>();  // after the first rows: 6 + 2 + 2 + 6 + 2 + 6
  bare_barrier();
#pragma unroll
  for (int i = 0; i < 3; ++i) x[i] = row_block(0, i);
  clear();
  int ks = 0;          // first step of the round that the loads of slot 3 are in
  bool fresh = false;  // the first round after another tile's stores
  for (;;) {
    const bool last = ks + 4 >= steps;  // the last round of this tile
    const Unit tile_unit = unit;
    const int tile_col = col0;
    const int live = tile_unit.expert < 0 ? 0 : tile_unit.rows;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      // rows(i + 1) have arrived for every wave, and every wave has read
      // rows(i - 1), whose slot the next loads fill
      __builtin_amdgcn_sched_barrier(0);
      if (s == 0 && fresh)  // the last tile's stores came in between
        wait_vmcnt<14 + STORES>();
      else if (s == 1 && fresh)
        wait_vmcnt<16 + STORES>();
      else if (s & 1)
        wait_vmcnt<16>();
      else
        wait_vmcnt<14>();
      bare_barrier();
      __builtin_amdgcn_sched_barrier(0);
      // The prepared scale dwords hold, at lane 16 c + n, chunk c of columns n
      // (byte 0, or 2 in odd steps) and 16 + n (byte 1 or 3).  Two swaps spread
      // the chunks of each half over the lanes that the instruction takes them
      // from, and a shift brings the lane's column to byte 0 or 2.
      if ((s & 1) == 0) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          wscale[nt][0] = wscale[nt][1] = st[s].bs[nt];
          swap16(wscale[nt][0], wscale[nt][1]);
          swap32(wscale[nt][0], wscale[nt][1]);
          wscale[nt][0] >>= 8 * r1;
          wscale[nt][1] >>= 8 * r1;
        }
      }
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        const int mt = i >> 1, h = i & 1;
        x[(i + 3) & 3] = i + 3 < 2 * MT ? row_block(s, i + 3) : row_block((s + 1) & 3, i + 3 - 2 * MT);
        if (64 * (mt >> 1) < live)  // 64 rows at a time: fewer conditions to keep
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
            acc[mt][nt] = mfma32_fp4_sel2(st[s].b[nt][h], x[i & 3], acc[mt][nt], wscale[nt][h], 2 * (s & 1),
                                          st[s].as[mt >> 1], 2 * (mt & 1) + h);
        __builtin_amdgcn_sched_barrier(0);
        load_part(ks, (s + 3) & 3, i);
      }
      if (s == 0) {
        ks += 4;
        if (last) {
          ks = 0;
          enter();
        }
      }
    }
    fresh = last;
    if (last) {
      if (wide_stores) {
        store(tile_unit, tile_col, std::true_type{});
      } else {
        store(tile_unit, tile_col, std::false_type{});
        wait_vmcnt<0>();
      }
      if (none) break;
      clear();
    }
  }
  wait_vmcnt<0>();  // no load may write to LDS that another workgroup has by then
}

}  // namespace mxfp4
