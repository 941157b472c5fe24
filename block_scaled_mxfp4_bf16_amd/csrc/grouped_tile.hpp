// The grouped product for groups of many rows (template; instantiated by
// grouped_kernels.hip): 128 rows x 256 weight rows per workgroup, two
// workgroups on a CU.
//
// The four waves share the 128 rows and split the columns, 64 each, so
//   - a block of weights is needed by one wave only and goes from memory to
//     its registers, four K steps ahead;
//   - the rows go through LDS, one 8 KiB slot per K step written directly by
//     the memory system, four slots in a ring; LDS then serves 40 KiB a step
//     and workgroup, where staging the weights as well would take 72 and make
//     LDS the bound;
//   - the weights are the first operand of the matrix instruction: a lane then
//     holds four neighbouring columns of one row and stores 8 bytes.
// Workgroups stay and walk over tiles; the loads run on into the next tile
// while the last steps and the stores of this one are under way.
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

template <bool GATED>
__global__ __launch_bounds__(256, 2) void grouped_tile_kernel(const GroupedArgs a, int n_tiles, int wide_stores) {
  constexpr int MT = 8, NT = 4;
  constexpr int BN = GATED ? 128 : 256;  // output columns of a tile
  constexpr int kNowhere = (int)0x80000000u;  // an offset that every buffer ends below
  __shared__ __attribute__((aligned(16))) uint8_t slot0[MT * 1024];
  __shared__ __attribute__((aligned(16))) uint8_t slot1[MT * 1024];
  __shared__ __attribute__((aligned(16))) uint8_t slot2[MT * 1024];
  __shared__ __attribute__((aligned(16))) uint8_t slot3[MT * 1024];
  const auto slot = [&](int s) -> uint8_t * { return s == 0 ? slot0 : (s == 1 ? slot1 : (s == 2 ? slot2 : slot3)); };

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane * 16, l4 = lane * 4;
  const int N = a.N, K = a.K;
  const int KS = (K + 127) >> 7;
  const int steps = (KS + 3) & ~3;  // steps past K load and add nothing
  const int gp = ((K >> 5) + 7) & ~7;
  const int b_bytes = (N >> 4) * K * 8;
  const int s_bytes = ((N + 255) >> 8) * 8 * gp * 32;
  const int out_cols = GATED ? N >> 1 : N;

  // Workgroup b runs on XCD b % 8.  Each XCD takes a contiguous range of the
  // items (unit, n tile), n tile fastest, so that an expert's weights and
  // rows stay in one L2.
  const int units = plan_entry(a, 0).expert;
  const int items = units * n_tiles;
  const int xcd = blockIdx.x & 7;
  const int stride = gridDim.x >> 3;
  const int end = (int)((int64_t)items * (xcd + 1) >> 3);
  int next_item = (int)((int64_t)items * xcd >> 3) + (blockIdx.x >> 3);
  if (next_item >= end) return;

  // What the loads of a tile need.  `none` (no tile left) has empty buffers.
  __amdgpu_buffer_rsrc_t a_rsrc, as_rsrc, b_rsrc, s_rsrc;
  int b_off, s_off;    // byte offsets of the wave's first group and its scales
  int b_off2, s_off2;  // the same of its second pair of groups (the up columns)
  Unit unit;           // of the tile that the loads are in
  int col0;            // its first output column of this wave
  bool none;

  auto enter = [&]() {
    none = next_item >= end;
    const int u = none ? 0 : next_item / n_tiles;
    const int n_tile = none ? 0 : next_item - u * n_tiles;
    next_item += stride;
    unit = plan_entry(a, 1 + u);
    const int tiles = none || unit.expert < 0 ? 0 : (unit.rows < 128 ? (unit.rows + 15) >> 4 : MT);
    const int64_t expert = unit.expert < 0 ? 0 : unit.expert;
    a_rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)(a.codes + (int64_t)unit.tile * KS * 1024), 0,
                                               tiles * KS * 1024, kRsrcWord3);
    as_rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)(a.scales + (int64_t)(unit.tile >> 2) * KS * 256), 0,
                                                ((tiles + 3) >> 2) * KS * 256, kRsrcWord3);
    b_rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)(a.Bw + expert * b_bytes), 0, tiles ? b_bytes : 0, kRsrcWord3);
    s_rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)(a.Bs + expert * s_bytes), 0, tiles ? s_bytes : 0, kRsrcWord3);
    col0 = n_tile * BN + wave * (BN / 4);
    const int g = col0 >> 4;
    const int up = GATED ? N >> 5 : 2;
    const bool ok1 = GATED ? g < (N >> 5) : g < (N >> 4);
    const bool ok2 = GATED ? ok1 : g + 2 < (N >> 4);
    b_off = ok1 ? g * K * 8 : kNowhere;
    b_off2 = ok2 ? (g + up) * K * 8 : kNowhere;
    s_off = ok1 ? (g >> 1) * gp * 32 : kNowhere;
    s_off2 = ok2 ? ((g + up) >> 1) * gp * 32 : kNowhere;
  };

  // Rows of step ks of the loads' tile into slot s: two of its eight blocks by
  // each wave.
  auto load_rows = [&](int ks, int s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * wave + i;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          a_rsrc, (__attribute__((address_space(3))) void *)(slot(s) + t * 1024), 16,
          uniform_off(ks < KS, (t * KS + ks) * 1024) + l16, 0, 0, 0);
    }
  };
  struct Stage {
    u32x4 b[NT];
    uint32_t as[2];
    uint32_t bs[2];  // of an even step and the next one; unused in odd stages
  };
  Stage st[4];
  auto load_weights = [&](int ks, int s) {
    const bool ok = ks < KS;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      st[s].b[nt] = __builtin_amdgcn_raw_buffer_load_b128(
          b_rsrc, uniform_off(ok, (nt < 2 ? b_off : b_off2) + (nt & 1) * K * 8 + ks * 1024) + l16, 0, 0);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      st[s].as[q] = __builtin_amdgcn_raw_buffer_load_b32(as_rsrc, uniform_off(ok, (q * KS + ks) * 256) + l4, 0, 0);
    if (s & 1) {
      // the weights' scales of this step and the one before, whose stage is
      // loaded but not yet in use; at an odd step the old ones are done with
#pragma unroll
      for (int q = 0; q < 2; ++q)
        st[s - 1].bs[q] = __builtin_amdgcn_raw_buffer_load_b32(
            s_rsrc, uniform_off(ks - 1 < KS, (q ? s_off2 : s_off) + (ks >> 1) * 256) + l4, 0, 0);
    }
  };
  auto row_block = [&](int s, int mt) { return *(const u32x4 *)(slot(s) + mt * 1024 + l16); };

  v4f acc[MT][NT];
  auto clear = [&]() {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = v4f{0.f, 0.f, 0.f, 0.f};
  };
  auto store = [&](const Unit &u, int col, auto wide) {
    const int rows = u.expert < 0 ? 0 : (u.rows < 128 ? u.rows : 128);
    const int ldc = (int)a.ldc * 2;
    const __amdgpu_buffer_rsrc_t c_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(a.C + (int64_t)u.row * a.ldc), 0, rows ? (rows - 1) * ldc + out_cols * 2 : 0, kRsrcWord3);
    const int at = (lane & 15) * ldc + (col + (lane >> 4) * 4) * 2;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const bool row_ok = 16 * mt + (lane & 15) < rows;
#pragma unroll
      for (int nt = 0; nt < (GATED ? NT / 2 : NT); ++nt) {
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = GATED ? gated_silu(acc[mt][nt][r], acc[mt][(nt + 2) % NT][r]) : acc[mt][nt][r];
        const bool ok = row_ok && col + 16 * nt < out_cols;
        const int off = off_or_oob(ok, at + 16 * mt * ldc + 32 * nt);
        const uint32_t lo = bf16x2_rne(v[0], v[1]), hi = bf16x2_rne(v[2], v[3]);
        if constexpr (decltype(wide)::value) {
          typedef uint32_t u32x2s __attribute__((ext_vector_type(2)));
          __builtin_amdgcn_raw_buffer_store_b64(u32x2s{lo, hi}, c_rsrc, off, 0, 0);
        } else {
          __builtin_amdgcn_raw_buffer_store_b16((uint16_t)lo, c_rsrc, off, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(lo >> 16), c_rsrc, off, 2, 0);
          __builtin_amdgcn_raw_buffer_store_b16((uint16_t)hi, c_rsrc, off, 4, 0);
          __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(hi >> 16), c_rsrc, off, 6, 0);
        }
      }
    }
  };

  // Loads go out in this order, each step's weights (6 loads, 8 in odd steps)
  // four steps and its rows (2 loads) three steps ahead:
  //   step i: rows(i + 3), weights(i + 4); step i + 1: rows(i + 4), ...
  // so at the start of step i the 16 newest loads came after rows(i + 1).
  // The scheduling barriers keep the compiler from mixing the steps' loads:
  // the load counter retires in issue order.
  u32x4 x[4];
  enter();
  load_rows(0, 0);
  __builtin_amdgcn_sched_barrier(0);
  load_weights(0, 0);
  __builtin_amdgcn_sched_barrier(0);
  load_weights(1, 1);
  __builtin_amdgcn_sched_barrier(0);
  load_rows(1, 1);
  __builtin_amdgcn_sched_barrier(0);
  load_weights(2, 2);
  __builtin_amdgcn_sched_barrier(0);
  load_rows(2, 2);
  __builtin_amdgcn_sched_barrier(0);
  load_weights(3, 3);
  __builtin_amdgcn_sched_barrier(0);
  wait_vmcnt<32>();
  bare_barrier();
#pragma unroll
  for (int i = 0; i < 3; ++i) x[i] = row_block(0, i);
  clear();
  int ks = 0;  // first step of the round that the loads of slot 3 are in
  for (;;) {
    const bool last = ks + 4 >= steps;  // the last round of this tile
    const Unit tile_unit = unit;
    const int tile_col = col0;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      // rows(i + 1) have arrived for every wave, and every wave has read
      // rows(i - 1), whose slot the next load fills
      __builtin_amdgcn_sched_barrier(0);
      wait_vmcnt<16>();
      bare_barrier();
      __builtin_amdgcn_sched_barrier(0);
      load_rows(s == 0 ? ks + 3 : ks + s - 1, (s + 3) & 3);
      if (s == 0) {
        ks += 4;
        if (last) {
          ks = 0;
          enter();
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        x[(mt + 3) & 3] = mt + 3 < MT ? row_block(s, mt + 3) : row_block((s + 1) & 3, mt + 3 - MT);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          acc[mt][nt] = mfma_fp4_sel2(st[s].b[nt], x[mt & 3], acc[mt][nt], st[s & 2].bs[nt >> 1], (nt & 1) + 2 * (s & 1),
                                      st[s].as[mt >> 2], mt & 3);
        __builtin_amdgcn_sched_barrier(0);
      }
      load_weights(ks + s, s);
    }
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
