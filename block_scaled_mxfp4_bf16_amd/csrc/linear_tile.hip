// The dense layer for many rows: 256 rows x 256 weight rows a workgroup, one on
// each CU.
//
// A K step of 128 is 32 blocks of 1 KiB, the 16 rows x 128 codes that the matrix
// instruction takes, written to LDS directly by the memory system, four steps in
// a ring, loaded up to four steps ahead; their scales lie beside them, two steps
// together.  Eight waves, 64 rows x 128 weight rows each, read every block from
// there while the products of the blocks before are under way.  So every
// line is taken in once a workgroup: 34 KiB a step for 256 x 256 outputs, where
// 128 x 256 tiles with their weights in registers take 48 for the same work.  One
// barrier a step, between its halves.
// Workgroups stay and walk over tiles; the loads run on into the next tile while
// the last steps and the epilogue of this one are under way.
//
// A step takes 0.7 to 0.8 us, of which the matrix units work 0.43 at 2.4 GHz and 0.5
// at the clock that they leave; without its loads it takes 0.67, without its products
// 0.43.  Median launches: 8192 x 4096 x 8192 with residual 158 us (least 154); gated
// 8192 x 16384 x 4096 with z kept 292 (277), where 402 MB of outputs, written by all
// CUs at a time, take a third, and up to 330 by where the buffers lie.  Starting the CUs
// up to 11 us apart so that these bursts spread changed nothing.
// The sums of two neighbouring blocks change places between lanes, after which a
// lane has 8 neighbouring columns of a row and four lanes 64 bytes of bf16.  (Turned
// in LDS, 8 rows x 64 columns a wave at a time, a tile's epilogue took 13 us for
// the 8 us of this form, most of it waiting for LDS.)
#include "linear_bounds.hpp"
#include "linear_epilogue.hpp"
#include "linear_internal.hpp"

namespace mxfp4 {

// Scale bytes `SA` and `SB` of the dwords.
template <int SA, int SB>
__device__ __forceinline__ v4f mfma_at(const u32x4 &a, const u32x4 &b, const v4f &c, uint32_t sa, uint32_t sb) {
  const v8i av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, SA, (int)sa, SB, (int)sb);
}
// ... of 16-row groups x and y in step s.
__device__ __forceinline__ v4f mfma_of(int x, int y, int s, const u32x4 &a, const u32x4 &b, const v4f &c, uint32_t sa,
                                       uint32_t sb) {
  switch ((x & 1) + 2 * (y & 1) + 4 * (s & 1)) {
    case 0: return mfma_at<0, 0>(a, b, c, sa, sb);
    case 1: return mfma_at<1, 0>(a, b, c, sa, sb);
    case 2: return mfma_at<0, 1>(a, b, c, sa, sb);
    case 3: return mfma_at<1, 1>(a, b, c, sa, sb);
    case 4: return mfma_at<2, 2>(a, b, c, sa, sb);
    case 5: return mfma_at<3, 2>(a, b, c, sa, sb);
    case 6: return mfma_at<2, 3>(a, b, c, sa, sb);
    default: return mfma_at<3, 3>(a, b, c, sa, sb);
  }
}

// From memory to LDS, 16 or 4 bytes a lane, lane after lane from `to` on.
__device__ __forceinline__ void block_to_lds(const __amdgpu_buffer_rsrc_t &r, uint8_t *to, int offset, int uniform) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)to, 16, offset, uniform, 0, 0);
}
__device__ __forceinline__ void scales_to_lds(const __amdgpu_buffer_rsrc_t &r, uint8_t *to, int offset, int uniform) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)to, 4, offset, uniform, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t sized(const void *base, int size) {
  return __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, size, kRsrcWord3);
}

template <bool GATED>
__global__ __launch_bounds__(512, 2) void linear_tile_kernel(const LinearArgs a, int m_tiles, int n_tiles) {
  constexpr int kSlot = 32 * 1024, kScales = 4096;
  constexpr int FI = 4, FK = 8;               // 16-row blocks of a wave: rows, weight rows
  constexpr int BN = GATED ? 128 : 256;       // output columns of a tile
  constexpr int kStores = GATED ? 8 : 16;     // of y, at least, by a wave and tile
  constexpr int kPreStores = 16;  // of the kept z
  __shared__ __attribute__((aligned(16))) uint8_t s0[kSlot], s1[kSlot], s2[kSlot], s3[kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t c0[kScales], c1[kScales];
  const auto slot = [&](int s) -> uint8_t * { return s == 0 ? s0 : (s == 1 ? s1 : (s == 2 ? s2 : s3)); };
  const auto scale_slot = [&](int s) -> uint8_t * { return s == 0 ? c0 : c1; };

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave & 3, wk = wave >> 2;  // the wave's 64 rows and 128 weight rows
  const int N = a.N, K = a.K;
  const int steps = tile_steps(K);  // those past K multiply zeros
  const int gp = ((K >> 5) + 7) & ~7;
  const int b_bytes = (N >> 4) * K * 8, s_bytes = ((N + 255) >> 8) * 8 * gp * 32;

  // Workgroup b runs on XCD b % 8.  Each XCD takes a run of tiles, blocks of 8 of
  // the rows with the columns outside, so that its 32 workgroups read 8 tiles of
  // rows and 4 of weights at a time.
  const int tiles = m_tiles * n_tiles;
  const int xcd = blockIdx.x & 7, stride = gridDim.x >> 3;
  const int end = (int)((int64_t)tiles * (xcd + 1) >> 3);
  int next = (int)((int64_t)tiles * xcd >> 3) + (blockIdx.x >> 3);
  if (next >= end) return;

  // What the loads of a tile need.  Past the last one the buffers have size 0.
  struct Tile {
    int m0, n0;  // first row and first output column
    const uint8_t *x, *xs;
    int x_size, xs_size, w_size, ws_size;
    int b_off[2], s_off;  // of the weight blocks that this wave loads
  };
  int none = 0;  // whether no tile was left for the last find()
  auto find = [&]() __attribute__((always_inline)) {
    Tile u;
    none = next >= end;
    const int t = none ? 0 : next;
    next += stride;
    const int block = t / (8 * n_tiles), in = t - block * 8 * n_tiles;
    const int high = m_tiles - 8 * block < 8 ? m_tiles - 8 * block : 8;
    const int nt = in / high;
    u.m0 = (8 * block + in - nt * high) * 256;
    u.n0 = nt * BN;
    const int rows = a.M - u.m0 < 256 ? a.M - u.m0 : 256;
    u.x = a.codes + (int64_t)(u.m0 >> 4) * K * 8;
    u.xs = a.scales + (int64_t)(u.m0 >> 5) * gp * 32;
    u.x_size = none ? 0 : ((rows + 15) >> 4) * K * 8;
    u.xs_size = none ? 0 : ((rows + 31) >> 5) * gp * 32;
    u.w_size = none ? 0 : b_bytes;
    u.ws_size = none ? 0 : s_bytes;
    // the wave's blocks 2 w and 2 w + 1 of 16; gated, of each 8 blocks the first
    // four are the gate's and the others their up rows; past the last group that one
    // again
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int b = 2 * wave + q;
      const int g = GATED ? ((b >> 2) & 1) * (N >> 5) + (u.n0 >> 4) + (b >> 3) * 4 + (b & 3) : (u.n0 >> 4) + b;
      u.b_off[q] = group_within(g, N >> 4) * K * 8;
    }
    const int g = GATED ? ((wave >> 1) & 1) * (N >> 6) + (u.n0 >> 5) + (wave >> 2) * 2 + (wave & 1) : (u.n0 >> 5) + wave;
    u.s_off = g * gp * 32;
    // The quotients come from the vector unit, and the compiler may leave all that
    // follows from them there, the loads' buffers among it.
    asm("" : "+s"(u.m0), "+s"(u.n0), "+s"(u.x), "+s"(u.xs), "+s"(u.b_off[0]), "+s"(u.b_off[1]), "+s"(u.s_off));
    asm("" : "+s"(u.x_size), "+s"(u.xs_size), "+s"(u.w_size), "+s"(u.ws_size));
    return u;
  };
  Tile cur = find();           // of the loads
  int row0 = cur.m0, col0 = cur.n0;  // of the products
  Tile after = find();         // the one after it
  int lk = 0;                  // step of the loads
  const int l16 = lane * 16, l4 = lane * 4, l_k = (lane >> 4) * 32;
  // Loads of step lk into a slot: this wave's two blocks of rows, its two of
  // weights, and of even steps its two blocks of scales.
  auto load_rows = [&](int to) __attribute__((always_inline)) {
    const int off = off_or_oob(lk * 128 + l_k < K, l16);  // chunks past K are zeros here, whatever the weights' are
#pragma unroll
    for (int q = 0; q < 2; ++q)
      block_to_lds(sized(cur.x, cur.x_size), slot(to) + (2 * wave + q) * 1024, off, (2 * wave + q) * K * 8 + lk * 1024);
  };
  auto load_weights = [&](int to) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      block_to_lds(sized(a.Bw, cur.w_size), slot(to) + (16 + 2 * wave + q) * 1024, l16, cur.b_off[q] + lk * 1024);
  };
  auto load_scales = [&](int to) __attribute__((always_inline)) {
    const bool ok = (lk >> 1) * 8 < gp;
    scales_to_lds(sized(cur.xs, ok ? cur.xs_size : 0), scale_slot(to) + wave * 256, l4, wave * gp * 32 + (lk >> 1) * 256);
    scales_to_lds(sized(a.Bs, ok ? cur.ws_size : 0), scale_slot(to) + 2048 + wave * 256, l4, cur.s_off + (lk >> 1) * 256);
  };
  // On to the next step, or the next tile; selects, since a branch would let the
  // compiler move the products into one of its ways.
  auto leave = [&](bool last) __attribute__((always_inline)) {
    lk = last ? 0 : lk + 1;
    cur.x = last ? after.x : cur.x;
    cur.xs = last ? after.xs : cur.xs;
    cur.x_size = last ? after.x_size : cur.x_size;
    cur.xs_size = last ? after.xs_size : cur.xs_size;
    cur.w_size = last ? after.w_size : cur.w_size;
    cur.ws_size = last ? after.ws_size : cur.ws_size;
    cur.b_off[0] = last ? after.b_off[0] : cur.b_off[0];
    cur.b_off[1] = last ? after.b_off[1] : cur.b_off[1];
    cur.s_off = last ? after.s_off : cur.s_off;
  };

  // A block is what the 16x16x128 instruction takes, lane after lane, and so is
  // a prepared scale dword: byte g + 2 o is that of group g of its 32 rows in step
  // o of its two.
  u32x4 xf[FI], wf[FK];
  auto read_weights = [&](int s, int x) __attribute__((always_inline)) { wf[x] = *(const u32x4 *)(slot(s) + (16 + 8 * wk + x) * 1024 + l16); };
  auto read_rows = [&](int s, int y) __attribute__((always_inline)) { xf[y] = *(const u32x4 *)(slot(s) + (4 * wi + y) * 1024 + l16); };
  uint32_t xs[2][FI / 2], ws[2][FK / 2];
  auto read_scales = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < FK / 2; ++n) ws[s][n] = *(const uint32_t *)(scale_slot(s) + 2048 + (4 * wk + n) * 256 + l4);
#pragma unroll
    for (int n = 0; n < FI / 2; ++n) xs[s][n] = *(const uint32_t *)(scale_slot(s) + (2 * wi + n) * 256 + l4);
  };

  v4f acc[FK][FI];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < FK; ++x)
#pragma unroll
      for (int y = 0; y < FI; ++y) acc[x][y] = v4f{0.f, 0.f, 0.f, 0.f};
  };

  // Half h of the step in slot s: the products of two of the wave's four row
  // blocks.  In the first the other two are read; in the second, after the barrier,
  // each block of weights is followed by the next step's in the same registers.
  // Between the products the loads go out: the barrier has freed slot s, which
  // takes the step four on, its rows at once and its weights in the next half.
  auto half_step = [&](int s, int h, int past) __attribute__((always_inline)) {
    const int sp = s >> 1, next = (s + 1) & 3;
#pragma unroll
    for (int x = 0; x < FK; ++x) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int y = 2 * h + q;
        acc[x][y] = mfma_of(x, y, s, wf[x], xf[y], acc[x][y], ws[sp][x >> 1], xs[sp][y >> 1]);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (h == 0) {
        if (x < 2) read_rows(s, 2 + x);
        if (x == 3) load_weights((s + 3) & 3);
        if (x == 5) leave(s == 0 && past >= 0);
      } else {
        read_weights(next, x);
        if (x < 2) read_rows(next, x);
        if (x == 2 && (s & 1) == 0) load_scales(sp);
        if (x == 4) load_rows(s);
        if (x == 6 && (s & 1) == 1) read_scales(next >> 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // A lane holds columns 4 g .. 4 g + 3, g = lane / 16, of a block's row lane % 16.
  // Swapping lanes 16 - 31 of one block's sums with lanes 0 - 15 of the next one's
  // (and 48 - 63 with 32 - 47) leaves it eight neighbouring columns: pieces 0, 2, 1
  // and 3 of the two blocks' 32 for g = 0 .. 3.
  auto neighbours = [&](int x, int y, float (&v)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t p = __float_as_uint(acc[x][y][i]), q = __float_as_uint(acc[x + 1][y][i]);
      swap16(p, q);
      v[i] = __uint_as_float(p);
      v[4 + i] = __uint_as_float(q);
    }
  };
  auto epilogue = [&](int row0, int col0) __attribute__((always_inline)) {
    // The lane's number is found anew for each tile, from a zero that the compiler
    // cannot see through: it would keep the offsets of every store through the
    // products otherwise, and has no registers for them.
    uint32_t zero = 0;
    asm volatile("" : "+s"(zero));
    const int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero));
    const int cols = GATED ? N >> 1 : N, half = N >> 1;
    const int rows = a.M - row0 < 256 ? a.M - row0 : 256;
    const int size = a.y_type == 2 ? 4 : 2;
    const int ldy = (int)a.ldy * size, ldr = (int)a.ld_res * size, ldp = (int)a.ld_pre * 2;
    const __amdgpu_buffer_rsrc_t y_rsrc =
        sized((uint8_t *)a.y + (int64_t)row0 * ldy, (rows - 1) * ldy + cols * size);
    const __amdgpu_buffer_rsrc_t r_rsrc =
        sized((const uint8_t *)a.residual + (int64_t)row0 * ldr, a.residual ? (rows - 1) * ldr + cols * size : 0);
    const __amdgpu_buffer_rsrc_t p_rsrc =
        sized((uint8_t *)a.pre + (int64_t)row0 * ldp, a.pre ? (rows - 1) * ldp + N * 2 : 0);
    const int piece = ((lane >> 5) & 1) | ((lane >> 3) & 2);
    constexpr int PAIRS = GATED ? 2 : 4;
    const auto column = [&](int pair) { return col0 + (GATED ? 64 : 128) * wk + 32 * pair + 8 * piece; };
    float bias[PAIRS][GATED ? 2 : 1][8];
    if (a.bias) {
#pragma unroll
      for (int pair = 0; pair < PAIRS; ++pair) {
        const int col = column(pair) < cols ? column(pair) : 0;
        load8(a.bias, a.bias_type, col, a.wide_bias, bias[pair][0]);
        if (GATED) load8(a.bias, a.bias_type, half + col, a.wide_bias, bias[pair][GATED ? 1 : 0]);
      }
      // waited for here: a load that seems to be under way when the next tile
      // begins would make its products wait for all others
#pragma unroll
      for (int pair = 0; pair < PAIRS; ++pair)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          asm volatile("" : "+v"(bias[pair][0][i]));
          if (GATED) asm volatile("" : "+v"(bias[pair][GATED ? 1 : 0][i]));
        }
    }
#pragma unroll
    for (int pair = 0; pair < PAIRS; ++pair) {
      const int col = column(pair);
      const bool col_ok = col < cols;
      const auto offset = [&](int y, int ld, int col_bytes) {
        const int row = 64 * wi + 16 * y + (lane & 15);
        return off_or_oob(col_ok && row < rows, row * ld + col_bytes);
      };
      // the residual of all four row blocks before the first is used
      Raw8 r[FI];
      if (a.residual) {
#pragma unroll
        for (int y = 0; y < FI; ++y) r[y] = load_raw8(r_rsrc, a.y_type, offset(y, ldr, col * size), a.line_y);
      }
#pragma unroll
      for (int y = 0; y < FI; ++y) {
        float z[8], up[8];
        neighbours(2 * pair, y, z);
        if (GATED) neighbours(4 + 2 * pair, y, up);
        if (a.bias) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            z[i] += bias[pair][0][i];
            if (GATED) up[i] += bias[pair][GATED ? 1 : 0][i];
          }
        }
        if (a.pre) {
          store8(p_rsrc, 0, offset(y, ldp, col * 2), z, a.line_pre);
          if (GATED) store8(p_rsrc, 0, offset(y, ldp, (half + col) * 2), up, a.line_pre);
        }
        activate8(a.act, z);
        if (GATED) {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] *= up[i];
        }
        if (a.residual) add_raw8(r[y], a.y_type, z);
        store8(y_rsrc, a.y_type, offset(y, ldy, col * size), z, a.line_y);
        __builtin_amdgcn_sched_barrier(0);  // few values at a time: the sums fill the registers
      }
    }
  };

  // The sums stay where they are: the compiler must not put products off past a
  // branch.
  auto hold = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < FK; ++x)
#pragma unroll
      for (int y = 0; y < FI; ++y) asm volatile("" : "+v"(acc[x][y]));
  };

#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if ((s & 1) == 0) load_scales(s >> 1);
    load_rows(s);
    if (s < 3) {
      load_weights(s);
      ++lk;
    }
  }
  wait_vmcnt<12>();  // after step 0: blocks of steps 1 to 3, 4 + 4 + 2, and scales, 2
  lds_barrier();
  const auto begin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < FK; ++x) read_weights(0, x);
    read_rows(0, 0);
    read_rows(0, 1);
    read_scales(0);
    clear();
  };
  begin();
  int fresh = 0;  // the first steps after another tile's stores, which may still be under way; 2: with z among them
  for (;;) {
    for (int ks = 0; ks < steps; ks += 4) {
      const int past = __builtin_amdgcn_readfirstlane(ks + 4 - steps);  // the tile's end
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        half_step(s, 0, past);
        // the next step's blocks, and its scales, have arrived for every wave, and
        // every wave has read this step's; 10 loads came after them
        if (s < 2) {
          hold();
          if (fresh == 2)
            wait_vmcnt<10 + kStores + kPreStores>();
          else if (fresh)
            wait_vmcnt<10 + kStores>();
          else
            wait_vmcnt<10>();
        } else {
          wait_vmcnt<10>();
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        half_step(s, 1, past);
      }
      hold();
      fresh = 0;
    }
    const bool more = !none;
    epilogue(row0, col0);
    if (!more) break;
    row0 = after.m0, col0 = after.n0;
    after = find();
    begin();  // the last step has read the operands too, but the epilogue needs their registers
    fresh = a.line_y && (!a.pre || a.line_pre) ? (a.pre ? 2 : 1) : 0;
    if (!fresh) wait_vmcnt<0>();  // more stores than are counted
  }
  wait_vmcnt<0>();  // no load may write to LDS that another workgroup has by then
}

hipError_t launch_linear_tile(const LinearArgs &a, hipStream_t stream) {
  const int cols = a.gated ? a.N / 2 : a.N, width = a.gated ? 128 : 256;
  const int m_tiles = (a.M + 255) / 256, n_tiles = (cols + width - 1) / width;
  if (a.gated)
    linear_tile_kernel<true><<<256, 512, 0, stream>>>(a, m_tiles, n_tiles);
  else
    linear_tile_kernel<false><<<256, 512, 0, stream>>>(a, m_tiles, n_tiles);
  return hipGetLastError();
}

}  // namespace mxfp4
