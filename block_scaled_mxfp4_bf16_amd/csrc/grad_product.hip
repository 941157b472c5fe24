// Products of a bf16 matrix with an MXFP4 matrix along its rows:
//   out[i, k] = sum_j P[i, j] * T[j, k]
// which is the gradient of the dense layer's input (P = dz, T = the weights)
// and, with P transposed in memory, of its weights (P = dz^T, T = Q(x)).
//
// T's scales belong to 32 neighbours along k, while the sum runs over j, so
// the scaled FP4 instruction cannot take T: its values become bf16, exactly (three
// significant bits; only those of 2^128 and more overflow), and the bf16
// instruction multiplies.
#include "linear_device.hpp"
#include "linear_internal.hpp"

namespace mxfp4 {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

// 16 bits of each of 4 rows x 16 columns of LDS, turned: lane 4 r + c of 16
// reads 8 bytes, columns 4 c .. 4 c + 3 of row r, and lane i receives column i
// of the four rows.
__device__ __forceinline__ u32x2 read_turned(const uint8_t *p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4 *)p));
}

__device__ __forceinline__ bf16x8 join(const u32x2 &a, const u32x2 &b) {
  return __builtin_bit_cast(bf16x8, u32x4{a.x, a.y, b.x, b.y});
}

// 16 bytes a lane from memory to LDS, lane after lane from `to` on.
__device__ __forceinline__ void load_to_lds(const __amdgpu_buffer_rsrc_t &r, uint8_t *to, int offset, int uniform) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)to, 16, offset, uniform, 0, 0);
}

// Eight codes -> eight bf16, the scale's exponent field applied.
__device__ __forceinline__ u32x4 bf16_of_codes(uint32_t w, float scale) {
  u32x4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return r;
}

// Place of 16-byte chunk c in row j of an LDS tile of `row_bytes` a row (a
// multiple of 256) that is written row by row and read turned.  LDS has 64 banks
// of 4 bytes; a turned read takes 32 lanes at once, 64 bytes of each of 4 rows, which
// lie in banks of their own so.  (32 bytes apart, they made twice the conflicts.)
__device__ __forceinline__ constexpr int turn_swizzle(int j) { return ((j & 3) << 2) | ((j >> 2) & 1); }
__device__ __forceinline__ int turned_at(int j, int c, int row_bytes) {
  return j * row_bytes + ((c ^ turn_swizzle(j)) << 4);
}
// The same for rows of 128 bytes of which 16 lanes read chunk c of 16 rows.
__device__ __forceinline__ constexpr int line_swizzle(int row) { return (row >> 1) & 7; }

// BI x BK outputs a workgroup of W waves, WI of them along i; 64 of j a stage,
// taken in two halves of two 16-deep steps.
//   P  goes through LDS as it is, written by the memory system: a ring of three
//      stages, loaded two stages ahead, whole 128-byte lines of its rows.
//   T  comes as codes, three halves ahead; each lane turns its 16 codes of one
//      row into bf16 and writes them to one of two LDS tiles, a half ahead of their
//      use.  So every code is converted once a workgroup, and the turned reads give
//      the operand's eight j of one k.
// The operands of a step are read while the step before multiplies; the one
// barrier of a half stands between its two steps, after which the next half's
// T and the next stage's P are there and the places of the last ones are free.
//
// 256 x 256 tiles with 8 waves, 8192 x 16384 x 4096: 790 us, 1.39 PFLOP/s, and
// transposed to f32 820 and 17 for the rows' quantization, 1.31 PFLOP/s; the
// library's bf16 product of these sizes takes 692 to 800.  Power bounds it: the
// matrix units are busy 75 % of the time at 1.88 GHz, and operands of zeros take
// 592 us.  P as the instruction's first operand takes 2.5 % less than T.  With 4
// waves of 128 x 128 outputs 840 us; waves 2 x 4 over i x k or 4 x 2: 806 and 808, and
// transposed 876 and 866.  One tile a workgroup and CU: a last round that is not full
// costs as much as one that is (k 4160 for 4096, 544 tiles for 512: 1034 us for 798).
// 128 x 128 tiles with 4 waves, where those are too few: 0.62 us a stage of which
// the products are 0.21; the latency of a stage's reads bounds it.
template <int BI, int BK, int W, int WI, bool TRANSPOSED>
__global__ __launch_bounds__(64 * W, W / 4) void grad_product_kernel(const GradProductArgs a, int i_tiles,
                                                                                     int k_tiles) {
  constexpr int WK = W / WI;
  constexpr int FI = BI / (32 * WI), FK = BK / (32 * WK);  // 32-wide operands of a wave
  constexpr int P_STAGE = BI * 128, T_HALF = BK * 64;       // bytes
  constexpr int P_LOADS = P_STAGE / (1024 * W);             // of 1 KiB, of a wave and stage
  constexpr int PUTS = BK / (16 * W);                       // dwords of codes of a lane and half: 8 of each
  constexpr int SIDES = BK / 128;                           // of 4 chunks of T's rows, a wave's worth of lanes
  static_assert(SIDES * 128 == BK && (PUTS == 2 || PUTS == 4) && P_LOADS % 4 == 0,
                "all threads share T; a fourth of P's loads a step");
  __shared__ __attribute__((aligned(16))) uint8_t p0[P_STAGE], p1[P_STAGE], p2[P_STAGE], t0[T_HALF], t1[T_HALF];
  const auto p_slot = [&](int s) -> uint8_t * { return s == 0 ? p0 : (s == 1 ? p1 : p2); };
  const auto t_slot = [&](int s) -> uint8_t * { return s == 0 ? t0 : t1; };

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroup b runs on XCD b % 8; each XCD takes a run of tiles, blocks of 8 of
  // i with k outside, so that what its workgroups read at a time is shared in L2.
  int it, kt;
  {
    const int tiles = i_tiles * k_tiles, b = blockIdx.x;
    const int per = tiles >> 3, rest = tiles & 7, x = b & 7;
    const int t = x * per + (x < rest ? x : rest) + (b >> 3);
    const int block = t / (8 * k_tiles), in = t - block * 8 * k_tiles;
    const int high = i_tiles - 8 * block < 8 ? i_tiles - 8 * block : 8;
    kt = in / high;
    it = 8 * block + in - kt * high;
  }
  const int i0 = it * BI, k0 = kt * BK;
  const int wi = (wave % WI) * 32 * FI, wk = (wave / WI) * 32 * FK;
  const int gp = ((a.K >> 5) + 7) & ~7;
  const int stages = (a.J + 63) >> 6;
  const int first = blockIdx.y * a.split_stages;
  const int last = first + a.split_stages < stages ? first + a.split_stages : stages;
  const auto sized = [](const void *base, int size) {
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, size, kRsrcWord3);
  };

  // P: the part of a stage's load n of this wave that a lane fetches.  The
  // place in LDS is lane * 16, so the lane picks the chunk that belongs there.
  const int ld2 = (int)a.ldp * 2;
  const int rows_i = a.I - i0 < BI ? a.I - i0 : BI;
  const uint16_t *p_base = TRANSPOSED ? a.P + i0 : a.P + (int64_t)i0 * a.ldp;
  constexpr int PC = TRANSPOSED ? BI / 8 : 8;  // chunks of a row in LDS
  constexpr int PR = 64 / PC;                  // rows of a load
  // The lane's row in load 0, and its chunk, which is the same in loads n and
  // n + PV.
  constexpr int PV = TRANSPOSED ? 4 : 2;
  const int pl_row = wave * P_LOADS * PR + lane / PC;
  int pl_off[PV], pl_j[PV];
#pragma unroll
  for (int v = 0; v < PV; ++v) {
    const int r = pl_row + v * PR;
    const int c = (lane % PC) ^ (TRANSPOSED ? turn_swizzle(r) : line_swizzle(r));
    pl_off[v] = pl_row * ld2 + c * 16;
    pl_j[v] = c * 8;
  }
  // The buffer of the stage that P's loads are in (of size 0 past the last), and
  // the lane's offsets; all of it is advanced a stage at a time, since products
  // of addresses between the matrix instructions take more cycles than those hide.
  const int j_end = a.J < last * 64 ? a.J : last * 64;
  const uint16_t *p_at = TRANSPOSED ? p_base + (int64_t)first * 64 * a.ldp : p_base + first * 64;
  int p_left = j_end - first * 64;  // of j
  int p_size, p_off[PV];
  auto enter_p = [&]() {
    if (TRANSPOSED) {
      const int rows = p_left < 64 ? p_left : 64;
      p_size = rows > 0 ? (rows - 1) * ld2 + rows_i * 2 : 0;
    } else {
      p_size = p_left > 0 ? (rows_i - 1) * ld2 + (p_left < 64 ? p_left : 64) * 2 : 0;
    }
#pragma unroll
    for (int v = 0; v < PV; ++v) p_off[v] = TRANSPOSED ? pl_off[v] : off_or_oob(pl_j[v] < p_left, pl_off[v]);
  };
  auto leave_p = [&]() {
    p_at += TRANSPOSED ? (int64_t)a.ldp * 64 : 64;
    p_left -= 64;
  };
  auto load_p = [&](int slot, int n) {
    load_to_lds(sized(p_at, p_size), p_slot(slot) + (wave * P_LOADS + n) * 1024, p_off[n % PV], n * PR * ld2);
  };

  // T: row lane % 16 of the half's 16-row group wave % 2, chunk lane / 16 of side
  // (wave / 2) % SIDES of the columns; where that leaves waves over, each takes 8
  // of the chunk's 16 bytes.
  struct Raw {
    uint32_t codes[PUTS];
    uint32_t scales;
  } raw[3];
  const int tg = wave & 1, side = (wave >> 1) % SIDES, t_part = (wave / (2 * SIDES)) * PUTS;
  const int tc = (lane >> 4) + 4 * side;
  const int t_high = ((k0 >> 7) + side) & 1;  // the scales of 8 groups lie together, 4 by 4
  const int t_row = tg * 16 + (lane & 15);
  const bool t_col = (k0 >> 5) + tc < (a.K >> 5);
  const int t_code_off = tg * a.K * 8 + ((k0 >> 5) + tc) * 256 + (lane & 15) * 16 + t_part * 4;
  const uint8_t *c_at = a.codes + (int64_t)first * 4 * a.K * 8, *s_at = a.scales + (int64_t)first * 2 * gp * 32;
  int t_left = j_end - first * 64, c_size, s_size;
  auto enter_t = [&]() {
    c_size = t_left > 16 ? 2 * a.K * 8 : (t_left > 0 ? a.K * 8 : 0);
    s_size = t_left > 0 ? gp * 32 : 0;
  };
  auto leave_t = [&]() {
    c_at += 2 * a.K * 8;
    s_at += gp * 32;
    t_left -= 32;
  };
  const int t_scale_off = off_or_oob(t_col, (k0 >> 8) * 256 + lane * 4), t_code_at = off_or_oob(t_col, t_code_off);
  auto load_t = [&](int q) {
    if constexpr (PUTS == 4) {
      const u32x4 c = __builtin_amdgcn_raw_buffer_load_b128(sized(c_at, c_size), t_code_at, 0, 0);
      raw[q].codes[0] = c.x, raw[q].codes[1] = c.y, raw[q].codes[2] = c.z, raw[q].codes[3] = c.w;
    } else {
      const u32x2 c = __builtin_amdgcn_raw_buffer_load_b64(sized(c_at, c_size), t_code_at, 0, 0);
      raw[q].codes[0] = c.x, raw[q].codes[1] = c.y;
    }
    raw[q].scales = __builtin_amdgcn_raw_buffer_load_b32(sized(s_at, s_size), t_scale_off, 0, 0);
  };
  // Places in LDS, as one address a lane for each pattern of the swizzle; the
  // rest is added as constants.
  int t_put[PUTS];
#pragma unroll
  for (int c = 0; c < PUTS; ++c) t_put[c] = turned_at(t_row, 4 * tc + t_part + c, BK * 2);
  auto put_t = [&](int q, int slot, int c) {
    const float scale = __uint_as_float(((raw[q].scales >> (8 * (tg + 2 * t_high))) & 0xFF) << 23);
    *(u32x4 *)(t_slot(slot) + t_put[c]) = bf16_of_codes(raw[q].codes[c], scale);
  };

  // Operands of a step: columns col + lane % 32, rows 8 * (lane / 32) .. + 7 of
  // the 16 from row j.  The swizzle of a turned read depends on the row modulo 8
  // (and so on whether it is the first or the second four) and works on the
  // operand's number modulo 4.
  const int tr_row = (lane >> 5) * 8 + ((lane & 15) >> 2);
  const int tr_col = ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
  int t_get[4][2], p_get[4][2];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c = (wk + 32 * n + tr_col) * 2, d = (wi + 32 * n + tr_col) * 2;
      t_get[n][q] = turned_at(tr_row + 4 * q, c >> 4, BK * 2) + (c & 15);
      if (TRANSPOSED) p_get[n][q] = turned_at(tr_row + 4 * q, d >> 4, BI * 2) + (d & 15);
    }
    const int row = wi + (lane & 31);
    if (!TRANSPOSED) p_get[n][0] = row * 128 + (((2 * n + (lane >> 5)) ^ line_swizzle(row)) << 4);
  }
  bf16x8 tf[2][FK], pf[2][FI];
  // Operand n (of FK + FI) of step `step` (0 .. 3) of the stage in slot p, half in slot t.
  auto read_operand = [&](int to, int step, int p, int t, int n) {
    static_assert(FK <= 4 && FI <= 4 && FK + FI <= FK * FI, "an address for each operand");
    if (n < FK) {
      const uint8_t *m = t_slot(t) + (step & 1) * 16 * BK * 2;
      tf[to][n] = join(read_turned(m + t_get[n][0]), read_turned(m + t_get[n][1]));
    } else if (TRANSPOSED) {
      const uint8_t *m = p_slot(p) + step * 16 * BI * 2;
      pf[to][n - FK] = join(read_turned(m + p_get[n - FK][0]), read_turned(m + p_get[n - FK][1]));
    } else {
      pf[to][n - FK] = *(const bf16x8 *)(p_slot(p) + p_get[step][0] + (n - FK) * 32 * 128);
    }
  };

  v16f acc[FK][FI];
#pragma unroll
  for (int x = 0; x < FK; ++x)
#pragma unroll
    for (int y = 0; y < FI; ++y)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.f;

  constexpr int MMA_SLOTS = FK * FI - FK * FI * 5 / 8;
  // One step: its products, and between them the reads of the next step's
  // operands, a fourth of the loads of stage + 2, and in the first step of a half
  // the conversion of the next half and the load of the one after the next two.
  auto step = [&](int S, int n_step) {  // S: the stage's slot; both known when compiled
    const int h = n_step >> 1, cur = n_step & 1, nxt = cur ^ 1;
    const int half = 2 * S + h;  // modulo 6
    const int next_step = (n_step + 1) & 3, next_p = n_step == 3 ? (S + 1) % 3 : S;
    const int next_t = (n_step & 1) ? (half + 1) & 1 : half & 1;
    constexpr int OPS = FK + FI, MMA = FK * FI;
#pragma unroll
    for (int m = 0; m < MMA; ++m) {
      if (m < OPS) read_operand(nxt, next_step, next_p, next_t, m);
      acc[m / FI][m % FI] =
          __builtin_amdgcn_mfma_f32_32x32x16_bf16(pf[cur][m % FI], tf[cur][m / FI], acc[m / FI][m % FI], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (cur == 0 && m >= MMA / 4 && m < MMA / 4 + PUTS) put_t((half + 1) % 3, (half + 1) & 1, m - MMA / 4);
      if (cur == 0 && m == MMA / 2) load_t((half + 1) % 3);
      if (cur == 0 && m == MMA / 2 + 1) leave_t();
      if (cur == 1 && m == MMA / 2 + 1) enter_t();
      if (m >= MMA * 5 / 8 && m < MMA * 5 / 8 + P_LOADS / 4)
        load_p((S + 2) % 3, n_step * (P_LOADS / 4) + m - MMA * 5 / 8);
      if (n_step == 3 && m == MMA * 6 / 8) leave_p();
      if (n_step == 3 && m == MMA * 7 / 8) enter_p();
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(FK * FI >= 4 && MMA_SLOTS >= P_LOADS / 4, "room for the loads between the products");

  if (first < last) {
    // before the loop: P of two stages, T of the first half, raw T of the next three
    enter_p();
    enter_t();
#pragma unroll
    for (int n = 0; n < P_LOADS; ++n) load_p(0, n);
    leave_p();
    enter_p();
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      load_t(q);
      leave_t();
      enter_t();
    }
#pragma unroll
    for (int n = 0; n < P_LOADS; ++n) load_p(1, n);
    leave_p();
    enter_p();
#pragma unroll
    for (int c = 0; c < PUTS; ++c) put_t(0, 0, c);
    load_t(0);
    leave_t();
    enter_t();
    wait_vmcnt<P_LOADS + 6>();  // the first stage's P
    __syncthreads();
#pragma unroll
    for (int n = 0; n < FK + FI; ++n) read_operand(0, 0, 0, 0, n);
    // three stages a round, those past the last of zeros: one way out of the
    // loop leaves the sums where they are
    for (int stage = first; stage < last; stage += 3) {
#pragma unroll
      for (int S = 0; S < 3; ++S) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          step(S, 2 * h);
          // T of the next half is written and, for the last half, P of the next
          // stage has arrived: 3 / 4 of a stage's loads of P and 4 of T came after
          if (h == 1)
            wait_vmcnt<P_LOADS / 4 * 3 + 4>();
          __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
          __builtin_amdgcn_sched_barrier(0);
          asm volatile("" ::: "memory");
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          __builtin_amdgcn_sched_barrier(0);
          step(S, 2 * h + 1);
        }
      }
    }
  }
  wait_vmcnt<0>();  // no load may write to LDS that is used from here on, or by another workgroup
  __syncthreads();

  // A lane holds column lane % 32 of a 32 x 32 block and rows 8 p + 4 * (lane / 32)
  // + r.  f32: 32 lanes store 128 bytes of a row.
  if (a.splits > 1 || a.out_type == 2) {
    float *const out = a.splits > 1 ? a.partial + (int64_t)blockIdx.y * a.I * a.K : (float *)a.out;
    const int64_t ld = a.splits > 1 ? a.K : a.ld_out;
#pragma unroll
    for (int y = 0; y < FI; ++y)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int i = i0 + wi + 32 * y + 8 * p + 4 * (lane >> 5);
        float *const row = out + i * ld + k0 + wk + (lane & 31);
#pragma unroll
        for (int x = 0; x < FK; ++x) {
          if (k0 + wk + 32 * x >= a.K) continue;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (i + r < a.I) row[r * ld + 32 * x] = acc[x][y][4 * p + r];
        }
      }
    return;
  }
  // 16 bits: 32 rows x 64 columns at a time through LDS, so that 8 lanes store 128
  // bytes of a row.
  uint16_t *const turn = (uint16_t *)p0 + wave * 32 * 64;
#pragma unroll
  for (int y = 0; y < FI; ++y)
#pragma unroll
    for (int xx = 0; xx < FK; xx += 2) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 8 * p + 4 * (lane >> 5) + r, col = 32 * x + (lane & 31);
            const float v = acc[xx + x][y][4 * p + r];
            turn[row * 64 + (((col >> 3) ^ (row & 7)) << 3) + (col & 7)] =
                a.out_type == 0 ? __builtin_bit_cast(uint16_t, (__bf16)v) : __builtin_bit_cast(uint16_t, (_Float16)v);
          }
      wave_lds_fence();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = 8 * q + (lane >> 3), c = lane & 7;
        const u32x4 d = *(const u32x4 *)(turn + row * 64 + ((c ^ (row & 7)) << 3));
        const int i = i0 + wi + 32 * y + row, k = k0 + wk + 32 * xx + 8 * c;
        if (i >= a.I || k >= a.K) continue;
        uint16_t *const to = (uint16_t *)a.out + i * a.ld_out + k;
        if (a.wide) {
          *(u32x4 *)to = d;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            to[2 * e] = (uint16_t)d[e];
            to[2 * e + 1] = (uint16_t)(d[e] >> 16);
          }
        }
      }
      wave_lds_fence();  // before the next columns
    }
}

// Few rows of P (32 * FI at most): reading T bounds it, and nothing waits at a
// barrier before the sums.  24 rows of 4096 x 4096: 5.3 us and 1.7 for the splits'
// sums; 256 x 256 tiles took 21.  64 columns a workgroup; its waves and the splits
// take every 32 of j in turn, D of them loaded ahead.  A lane turns one chunk of
// 32 codes into bf16 in its wave's own 4 KiB of LDS, P's rows go straight to
// registers.  The waves' sums meet in LDS, in wave order.
constexpr int kFewWaves = 8;
template <int FI, int D>
__global__ __launch_bounds__(64 * kFewWaves) void grad_few_kernel(const GradProductArgs a) {
  constexpr int W = kFewWaves;
  __shared__ __attribute__((aligned(16))) float red[W][2][16][64];  // and before that the waves' tiles of T
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k0 = blockIdx.x * 64;
  const int G = a.K >> 5, gp = (G + 7) & ~7;
  const int units = (a.J + 31) >> 5;
  uint8_t *const tile = (uint8_t *)red + wave * 4096;

  // T: row lane % 16 of group lane / 32, chunk (lane / 16) % 2
  const int tg = lane >> 5, tc = (k0 >> 5) + ((lane >> 4) & 1), tr = lane & 15;
  const bool t_col = tc < G;
  const int t_bytes = ((a.J + 15) >> 4) * a.K * 8, s_bytes = ((a.J + 31) >> 5) * gp * 32;
  const __amdgpu_buffer_rsrc_t c_rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)a.codes, 0, t_bytes, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t s_rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)a.scales, 0, s_bytes, kRsrcWord3);
  const int c_off = off_or_oob(t_col, tg * a.K * 8 + tc * 256 + tr * 16);
  const int s_off = off_or_oob(t_col, (tc >> 3) * 256 + (tr << 2) + ((tc & 3) << 6));
  const int s_shift = 8 * (tg + 2 * ((tc >> 2) & 1));
  const int ld2 = (int)a.ldp * 2;
  const __amdgpu_buffer_rsrc_t p_rsrc =
      __builtin_amdgcn_make_buffer_rsrc((void *)a.P, 0, (a.I - 1) * ld2 + a.J * 2, kRsrcWord3);
  const int p_j = 8 * (lane >> 5);
  int p_off[FI];
#pragma unroll
  for (int y = 0; y < FI; ++y) {
    const int i = 32 * y + (lane & 31);
    p_off[y] = off_or_oob(i < a.I, i * ld2 + p_j * 2);
  }

  struct Stage {
    u32x4 codes;
    uint32_t scale;
    u32x4 p[2][FI];
  } st[D];
  auto load = [&](int q, int unit) {
    // past the last unit the lanes' offsets alone say so: with a uniform part of
    // 2^31 the sum of the two would be small again
    const bool ok = unit < units;
    const int u = ok ? unit : 0;
    st[q].codes = __builtin_amdgcn_raw_buffer_load_b128(c_rsrc, off_or_oob(ok, c_off), u * 2 * a.K * 8, 0);
    st[q].scale =
        __builtin_amdgcn_raw_buffer_load_b32(s_rsrc, off_or_oob(ok && 32 * u + 16 * tg < a.J, s_off), u * gp * 32, 0);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int y = 0; y < FI; ++y)
        st[q].p[s][y] = __builtin_amdgcn_raw_buffer_load_b128(
            p_rsrc, off_or_oob(ok && 32 * u + 16 * s + p_j < a.J, p_off[y]), u * 64 + s * 32, 0);
  };
  const auto place = [](int j, int c) { return j * 128 + ((c ^ (((j & 2) << 1) | ((j >> 2) & 1))) << 4); };
  const int tr_row = (lane >> 5) * 8 + ((lane & 15) >> 2);
  const int tr_col = (((lane >> 4) & 1) * 16 + (lane & 3) * 4) * 2;

  v16f acc[2][FI];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < FI; ++y)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.f;
  auto compute = [&](int q) {
    const float scale = __uint_as_float(((st[q].scale >> s_shift) & 0xFF) << 23);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *(u32x4 *)(tile + place(tg * 16 + tr, 4 * ((lane >> 4) & 1) + c)) = bf16_of_codes(st[q].codes[c], scale);
    wave_lds_fence();
    bf16x8 t[2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = 16 * s + tr_row, c = 64 * x + tr_col;
        t[s][x] = join(read_turned(tile + place(j, c >> 4) + (c & 15)), read_turned(tile + place(j + 4, c >> 4) + (c & 15)));
      }
    wave_lds_fence();  // before the next unit's codes
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < FI; ++y)
          acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, st[q].p[s][y]), t[s][x], acc[x][y],
                                                              0, 0, 0);
  };

  const int stride = W * gridDim.y, first = blockIdx.y * W + wave;
#pragma unroll
  for (int q = 0; q < D; ++q) load(q, first + q * stride);
  // units past the last are zeros; the last round loads nothing
  int u = first;
  for (; u - wave + D * stride < units; u += D * stride)
#pragma unroll
    for (int q = 0; q < D; ++q) {
      compute(q);
      load(q, u + (D + q) * stride);
    }
#pragma unroll
  for (int q = 0; q < D; ++q) compute(q);

  const bool split = gridDim.y > 1;
#pragma unroll
  for (int y = 0; y < FI; ++y) {
    if (32 * y >= a.I) break;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int r = 0; r < 16; ++r) red[wave][x][r][lane] = acc[x][y][r];
    __syncthreads();
    const int row = threadIdx.x >> 4, c = (threadIdx.x & 15) * 4;
    const int i = 32 * y + row, k = k0 + c;
    if (i < a.I && k < a.K) {
      const auto part = [&](int w) {
        return *(const v4f *)&red[w][c >> 5][4 * (row >> 3) + (row & 3)][((row >> 2) & 1) * 32 + (c & 31)];
      };
      v4f v = part(0);
#pragma unroll
      for (int w = 1; w < W; ++w) v += part(w);
      if (split)
        *(v4f *)(a.partial + ((int64_t)blockIdx.y * a.I + i) * a.K + k) = v;
      else
        store4(a.out, a.out_type, (int64_t)i * a.ld_out + k, v, a.wide4);
    }
  }
}

// The splits' sums, in order.
__global__ __launch_bounds__(256) void join_splits_kernel(const GradProductArgs a) {
  const int64_t quads = (int64_t)a.I * (a.K >> 2);
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (q >= quads) return;
  const int64_t i = q / (a.K >> 2);
  const int k = (int)(q - i * (a.K >> 2)) * 4;
  v4f v = *(const v4f *)(a.partial + i * a.K + k);
  for (int s = 1; s < a.splits; ++s) v += *(const v4f *)(a.partial + ((int64_t)s * a.I + i) * a.K + k);
  store4(a.out, a.out_type, i * a.ld_out + k, v, a.wide4);
}

namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a product is done: the form, and over how many workgroups the sum of one
// tile is split.
struct Plan {
  enum { kFew, kTile128, kTile256 } form;
  int splits, split_stages;
};

// Splits of `units` of j for `tiles` tiles: until every CU has a workgroup, and
// no fewer than `least` units each.
int64_t split_count(int64_t tiles, int64_t units, int64_t least) {
  const int64_t want = cdiv(256, tiles), most = units / least;
  return want < most ? (want < 1 ? 1 : want) : (most < 1 ? 1 : most);
}

Plan plan_of(int64_t I, int64_t J, int64_t K, bool transposed) {
  Plan p{Plan::kTile256, 1, 0};
  if (!transposed && I <= 128) {
    p.form = Plan::kFew;
    p.splits = (int)split_count(cdiv(K, 64), cdiv(J, 32), kFewWaves * 2);
    return p;
  }
  const int64_t stages = cdiv(J, 64);
  int64_t tiles = cdiv(I, 256) * cdiv(K, 256);
  if (tiles < 192) {
    p.form = Plan::kTile128;
    tiles = cdiv(I, 128) * cdiv(K, 128);
  }
  p.split_stages = (int)(cdiv(stages, 3) * 3);  // rounds of three stages
  if (p.form != Plan::kTile128) return p;
  // 128 x 128 tiles take 0.62 us a stage while two workgroups fit on every CU.  A
  // split costs its launch and what crosses the chiplets' caches, 5 us, and the
  // partial sums' way to memory and back, at 4 MB a us.  (Whole and in three:
  // 771 rows of 2112 x 704, 13 stages, 16.1 and 22.0 us a call; 3136 rows, 49
  // stages, 38.8 and 30.0.  256 rows of 4096 x 4096, 64 stages: 40.7 whole, 22.3 in
  // four.)
  double best = 0;
  for (int s = 1; s <= 16 && 3 * (s - 1) < stages; ++s) {
    const int64_t per = cdiv(cdiv(stages, s), 3) * 3;
    const double rounds = tiles * s > 512 ? tiles * s / 512.0 : 1.0;
    const double t = 0.62 * per * rounds + (s > 1 ? 5 + s * (double)I * K * 8 / 4e6 : 0);
    if (s > 1 && t >= best) continue;
    best = t;
    p.split_stages = (int)per;
    p.splits = (int)cdiv(stages, per);
  }
  if (p.splits < 1) p.splits = 1;
  return p;
}

template <int BI, int BK, int W, int WI, bool TRANSPOSED>
void run_tiles(const GradProductArgs &a, hipStream_t stream) {
  const int i_tiles = (int)cdiv(a.I, BI), k_tiles = (int)cdiv(a.K, BK);
  const dim3 grid((unsigned)(i_tiles * k_tiles), a.splits);
  grad_product_kernel<BI, BK, W, WI, TRANSPOSED><<<grid, 64 * W, 0, stream>>>(a, i_tiles, k_tiles);
}

}  // namespace

size_t grad_product_workspace_bytes(int64_t I, int64_t J, int64_t K, bool transposed) {
  const Plan p = plan_of(I, J, K, transposed);
  return p.splits > 1 ? (size_t)p.splits * (size_t)I * (size_t)K * 4 : 0;
}

hipError_t launch_grad_product(GradProductArgs a, hipStream_t stream) {
  const Plan p = plan_of(a.I, a.J, a.K, a.transposed);
  a.splits = p.splits;
  a.split_stages = p.split_stages;
  if (p.form == Plan::kFew) {
    const dim3 grid((unsigned)cdiv(a.K, 64), a.splits);
    if (a.I <= 32)
      grad_few_kernel<1, 4><<<grid, 64 * kFewWaves, 0, stream>>>(a);
    else if (a.I <= 64)
      grad_few_kernel<2, 3><<<grid, 64 * kFewWaves, 0, stream>>>(a);
    else
      grad_few_kernel<4, 2><<<grid, 64 * kFewWaves, 0, stream>>>(a);
  } else if (p.form == Plan::kTile128) {
    if (a.transposed)
      run_tiles<128, 128, 4, 2, true>(a, stream);
    else
      run_tiles<128, 128, 4, 2, false>(a, stream);
  } else if (a.transposed) {
    run_tiles<256, 256, 8, 4, true>(a, stream);
  } else {
    run_tiles<256, 256, 8, 2, false>(a, stream);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits <= 1) return e;
  const int64_t quads = (int64_t)a.I * (a.K / 4);
  join_splits_kernel<<<(unsigned)((quads + 255) / 256), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace mxfp4
