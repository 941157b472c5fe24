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

// Place of 16-byte chunk c in row j of an LDS tile of `row_bytes` a row that is
// written row by row and read turned: 8 rows' chunks c lie in other banks, and so
// do the two chunks of 4 rows that a turned read takes.
__device__ __forceinline__ int turned_at(int j, int c, int row_bytes) {
  return j * row_bytes + ((c ^ (((j & 3) << 1) | ((j >> 2) & 1))) << 4);
}

// BI x BK outputs a workgroup of 4 waves, WI of them along i; 64 of j a stage,
// taken in two halves of two 16-deep steps.
//   P  goes through LDS as it is, written by the memory system: a ring of three
//      stages, loaded two stages ahead, whole 128-byte lines of its rows.
//   T  comes as codes, 17 bytes a lane and half, three halves ahead; each lane
//      turns its 32 codes of one row into bf16 and writes them to one of two
//      LDS tiles, a half ahead of their use.  So every code is converted once a
//      workgroup, and the turned reads give the operand's eight j of one k.
// The operands of a step are read while the step before multiplies; the one
// barrier of a half stands between its two steps, after which the next half's
// T and the next stage's P are there and the places of the last ones are free.
template <int BI, int BK, int WI, bool TRANSPOSED>
__global__ __launch_bounds__(256, BI * BK > 128 * 128 ? 1 : 2) void grad_product_kernel(const GradProductArgs a, int i_tiles,
                                                                                     int k_tiles) {
  constexpr int WK = 4 / WI;
  constexpr int FI = BI / (32 * WI), FK = BK / (32 * WK);  // 32-wide operands of a wave
  constexpr int P_STAGE = BI * 128, T_HALF = BK * 64;       // bytes
  constexpr int P_LOADS = P_STAGE / 4096;                   // of 1 KiB, of a wave and stage
  static_assert(BK == 256 && P_LOADS % 4 == 0, "a thread a chunk of T, a fourth of P's loads a step");
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
  // The lane's row and chunk of load 0; for transposed rows the chunk of the
  // loads n and n + 4 is the same.
  constexpr int PV = TRANSPOSED ? 4 : 1;
  const int pl_row = wave * P_LOADS * PR + lane / PC;
  int pl_off[PV], pl_j = 0;
#pragma unroll
  for (int v = 0; v < PV; ++v) {
    const int r = pl_row + v * PR;
    const int c = (lane % PC) ^ (TRANSPOSED ? ((r & 3) << 1) | ((r >> 2) & 1) : r & 7);
    pl_off[v] = pl_row * ld2 + c * 16;
    pl_j = c * 8;
  }
  auto load_p = [&](int stage, int slot, int n) {
    uint8_t *to = p_slot(slot) + (wave * P_LOADS + n) * 1024;
    if (TRANSPOSED) {
      const int left = stage < last ? a.J - stage * 64 : 0;
      const int rows = left < 64 ? left : 64;
      const __amdgpu_buffer_rsrc_t rs =
          sized(p_base + (int64_t)(left > 0 ? stage * 64 : 0) * a.ldp, left > 0 ? (rows - 1) * ld2 + rows_i * 2 : 0);
      load_to_lds(rs, to, pl_off[n % PV], n * PR * ld2);
    } else {
      const __amdgpu_buffer_rsrc_t rs = sized(p_base, stage < last ? (rows_i - 1) * ld2 + a.J * 2 : 0);
      load_to_lds(rs, to, off_or_oob(stage * 64 + pl_j < a.J, pl_off[0]), n * PR * ld2 + stage * 128);
    }
  };

  // T: row lane % 16 of the half's 16-row group wave % 2, chunk lane / 16 of the
  // columns' half wave / 2.
  struct Raw {
    u32x4 codes;
    uint32_t scales;
  } raw[3];
  const int tg = wave & 1, tc = (lane >> 4) + 4 * (wave >> 1);
  const int t_row = tg * 16 + (lane & 15);
  const bool t_col = (k0 >> 5) + tc < (a.K >> 5);
  const int t_code_off = tg * a.K * 8 + ((k0 >> 5) + tc) * 256 + (lane & 15) * 16;
  auto load_t = [&](int half, int q) {
    const int j0 = half * 32;
    const int left = half < 2 * last ? a.J - j0 : 0;
    const int groups = left <= 0 ? 0 : (left > 16 ? 2 : 1);
    const int64_t at = left > 0 ? half : 0;
    const __amdgpu_buffer_rsrc_t rc = sized(a.codes + at * 2 * a.K * 8, groups * a.K * 8);
    const __amdgpu_buffer_rsrc_t rs = sized(a.scales + at * gp * 32, left > 0 ? gp * 32 : 0);
    raw[q].codes = __builtin_amdgcn_raw_buffer_load_b128(rc, off_or_oob(t_col, t_code_off), 0, 0);
    raw[q].scales = __builtin_amdgcn_raw_buffer_load_b32(rs, off_or_oob(t_col && tg < groups, (k0 >> 5) * 32 + lane * 4), 0, 0);
  };
  // Places in LDS, as one address a lane for each pattern of the swizzle; the
  // rest is added as constants.
  int t_put[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) t_put[c] = turned_at(t_row, 4 * tc + c, BK * 2);
  auto put_t = [&](int q, int slot, int c) {
    const float scale = __uint_as_float(((raw[q].scales >> (8 * (tg + 2 * (wave >> 1)))) & 0xFF) << 23);
    *(u32x4 *)(t_slot(slot) + t_put[c]) = bf16_of_codes(raw[q].codes[c], scale);
  };

  // Operands of a step: columns col + lane % 32, rows 8 * (lane / 32) .. + 7 of
  // the 16 from row j.  The swizzle of a turned read depends on the row modulo 8
  // (and so on whether it is the first or the second four) and on whether the
  // column is an even or odd multiple of 32.
  const int tr_row = (lane >> 5) * 8 + ((lane & 15) >> 2);
  const int tr_col = ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
  int t_get[2][2], p_get[4];
#pragma unroll
  for (int odd = 0; odd < 2; ++odd)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c = (wk + 32 * odd + tr_col) * 2;
      t_get[odd][q] = turned_at(tr_row + 4 * q, c >> 4, BK * 2) + (c & 15);
      const int d = (wi + 32 * odd + tr_col) * 2;
      if (TRANSPOSED) p_get[2 * odd + q] = turned_at(tr_row + 4 * q, d >> 4, BI * 2) + (d & 15);
    }
  if (!TRANSPOSED)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int row = wi + (lane & 31), c = s * 2 + (lane >> 5);
      p_get[s] = row * 128 + ((c ^ (row & 7)) << 4);
    }
  bf16x8 tf[2][FK], pf[2][FI];
  // Operand n (of FK + FI) of step `step` (0 .. 3) of the stage in slot p, half in slot t.
  auto read_operand = [&](int to, int step, int p, int t, int n) {
    if (n < FK) {
      const uint8_t *m = t_slot(t) + (step & 1) * 16 * BK * 2 + (n >> 1) * 128;
      tf[to][n] = join(read_turned(m + t_get[n & 1][0]), read_turned(m + t_get[n & 1][1]));
    } else if (TRANSPOSED) {
      const int y = n - FK;
      const uint8_t *m = p_slot(p) + step * 16 * BI * 2 + (y >> 1) * 128;
      pf[to][y] = join(read_turned(m + p_get[2 * (y & 1)]), read_turned(m + p_get[2 * (y & 1) + 1]));
    } else {
      pf[to][n - FK] = *(const bf16x8 *)(p_slot(p) + p_get[step] + (n - FK) * 32 * 128);
    }
  };

  v16f acc[FK][FI];
#pragma unroll
  for (int x = 0; x < FK; ++x)
#pragma unroll
    for (int y = 0; y < FI; ++y)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.f;

  // One step: its products, and between them the reads of the next step's
  // operands, a fourth of the loads of stage + 2, and in the first step of a half
  // the conversion of the next half and the load of the one after the next two.
  auto step = [&](int stage, int S, int n_step) {  // S = the stage's slot, all but `stage` known when compiled
    const int h = n_step >> 1, cur = n_step & 1, nxt = cur ^ 1;
    const int half = 2 * S + h;  // modulo 6
    const int next_step = (n_step + 1) & 3, next_p = n_step == 3 ? (S + 1) % 3 : S;
    const int next_t = (n_step & 1) ? (half + 1) & 1 : half & 1;
    constexpr int OPS = FK + FI, MMA = FK * FI;
#pragma unroll
    for (int m = 0; m < MMA || m < OPS; ++m) {
      if (m < OPS) read_operand(nxt, next_step, next_p, next_t, m);
      if (m < MMA)
        acc[m / FI][m % FI] =
            __builtin_amdgcn_mfma_f32_32x32x16_bf16(tf[cur][m / FI], pf[cur][m % FI], acc[m / FI][m % FI], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (cur == 0 && m >= 4 && m < 8) put_t((half + 1) % 3, (half + 1) & 1, m - 4);
      if (cur == 0 && m == 8) load_t(2 * stage + h + 4, (half + 1) % 3);
      if (m >= 10 && m < 10 + P_LOADS / 4) load_p(stage + 2, (S + 2) % 3, n_step * (P_LOADS / 4) + m - 10);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(FK * FI >= 10 + P_LOADS / 4, "room for the loads between the products");

  if (first < last) {
    // before the loop: P of two stages, T of the first half, raw T of the next three
#pragma unroll
    for (int n = 0; n < P_LOADS; ++n) load_p(first, 0, n);
    load_t(2 * first, 0);
    load_t(2 * first + 1, 1);
    load_t(2 * first + 2, 2);
#pragma unroll
    for (int n = 0; n < P_LOADS; ++n) load_p(first + 1, 1, n);
#pragma unroll
    for (int c = 0; c < 4; ++c) put_t(0, 0, c);
    load_t(2 * first + 3, 0);
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
          step(stage + S, S, 2 * h);
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
          step(stage + S, S, 2 * h + 1);
        }
      }
    }
    wait_vmcnt<0>();  // no load may write to LDS that another workgroup has by then
  }

#pragma unroll
  for (int y = 0; y < FI; ++y) {
    const int i = i0 + wi + 32 * y + (lane & 31);
    if (i >= a.I) continue;
#pragma unroll
    for (int x = 0; x < FK; ++x)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int k = k0 + wk + 32 * x + 8 * p + 4 * (lane >> 5);
        if (k >= a.K) continue;
        const v4f v = {acc[x][y][4 * p], acc[x][y][4 * p + 1], acc[x][y][4 * p + 2], acc[x][y][4 * p + 3]};
        if (a.splits > 1)
          *(v4f *)(a.partial + ((int64_t)blockIdx.y * a.I + i) * a.K + k) = v;
        else
          store4(a.out, a.out_type, (int64_t)i * a.ld_out + k, v, a.wide);
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
  store4(a.out, a.out_type, i * a.ld_out + k, v, a.wide);
}

// Workgroups that split the sum of one tile: until every CU has one, while
// each keeps 256 of j.
static int64_t splits_of(int64_t I, int64_t J, int64_t K) {
  const int64_t tiles = ((I + 255) / 256) * ((K + 255) / 256), most = J / 256;
  const int64_t want = 256 / tiles;
  const int64_t s = want < most ? want : most;
  return s < 1 ? 1 : s;
}

size_t grad_product_workspace_bytes(int64_t I, int64_t J, int64_t K) {
  const int64_t s = splits_of(I, J, K);
  return s > 1 ? (size_t)s * (size_t)I * (size_t)K * 4 : 0;
}

hipError_t launch_grad_product(GradProductArgs a, hipStream_t stream) {
  const int stages = (a.J + 63) / 64;
  const int64_t want = splits_of(a.I, a.J, a.K);
  a.split_stages = (int)((stages + want - 1) / want);
  a.splits = a.split_stages > 0 ? (stages + a.split_stages - 1) / a.split_stages : 1;
  const int i_tiles = (a.I + 255) / 256, k_tiles = (a.K + 255) / 256;
  const dim3 grid((unsigned)(i_tiles * k_tiles), a.splits);
  if (a.transposed)
    grad_product_kernel<256, 256, 2, true><<<grid, 256, 0, stream>>>(a, i_tiles, k_tiles);
  else
    grad_product_kernel<256, 256, 2, false><<<grid, 256, 0, stream>>>(a, i_tiles, k_tiles);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits <= 1) return e;
  const int64_t quads = (int64_t)a.I * (a.K / 4);
  join_splits_kernel<<<(unsigned)((quads + 255) / 256), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace mxfp4
