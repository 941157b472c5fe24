// Products of a few rows with MXFP4 weights, the activations unquantized:
//   y[r, n] = sum_k x[r, k] * e2m1(code[n, k]) * 2^(s[n, k / 32] - 127)
// and its gated form, silu(first half of the columns) * (second half).
//
// Reading the weights bounds it: N * K * 17/32 bytes against 2 * M * N * K
// flops.  A wave takes 16 columns x 128 elements of K at a time, one 16-byte
// load per lane (the prepared layout makes that 1 KiB contiguous), converts
// the codes to 16-bit floats with the hardware's scaled convert and feeds
// the 16x16x32 matrix instruction, whose 16 rows serve every M up to 16 at
// the same price.  The converts (16 per KiB) and the products (4 per KiB)
// leave the vector units idle most of the time at the rate that memory
// delivers, so there is nothing to win from a separate dot-product form for
// one row.
//
// Lane l of the load holds column l % 16 and group 4 * step + l / 16: all 32
// elements of one group, so one scale per lane.
//   bf16 rows  the convert applies the scale: e2m1 * 2^e is exact in bf16 (down
//              to 2^-128: subnormals count; beyond 2^128 see `compute`).  Product i takes elements 8i..8i+7 of the lane's group.
//   f32 rows   as bf16, with x cut into three bf16 parts of 8 significand
//              bits each: hi + mid + lo = x exactly down to the last bit of
//              bf16's subnormals, 2^-133, so that the only rounding is that of
//              the f32 sums, as in a product of f32 by f32.
//   f16 rows   a scaled weight may leave f16's range, so the codes are
//              converted unscaled and the f32 sum of each group is scaled
//              instead.  That needs products that stay within one group: the
//              four dwords of the lanes of a column are transposed over the
//              four lane quarters with two kinds of lane swaps, after which
//              product i takes the whole of group 4 * step + i.
// The waves of a workgroup split K and add their tiles through LDS in wave
// order; sums are f32, rounded once to y's type.
//
// Measured, a call among others, weights partly in the caches: 32 expert rows of
// 4096 x 2048, gated, 22.5 us, 5.2 TB/s of weights; one row of 7168 x 7168 6.3 us,
// 4.4 TB/s with the launch; the kernel of one row of 4096 x 512 2.9 us, a launch and
// one round of loads.  f32 rows, three products a step, in a graph over fresh
// weights: one row of 7168 x 7168 17.3 us, 32 expert rows 40.8; f16 rows 8.8 and 25.9,
// bf16 rows there 6.8 and 23.7.
#include <type_traits>

#include "experts_device.hpp"
#include "experts_internal.hpp"

namespace mxfp4 {

namespace {

enum { kBf16 = 0, kF16 = 1, kF32 = 2 };

// Bits of the largest scale, as f32, with which bf16 holds every weight (6 *
// 2^125), and of the scale that stands for NaN.
constexpr uint32_t kLargestScale = 252u << 23, kNanScale = 255u << 23;

// Eight weights of one dword of codes as bf16, scaled by a power of two.
__device__ __forceinline__ bf16x8 weights_bf16(uint32_t w, float scale) {
  union {
    bf16x2 h[4];
    bf16x8 v;
  } u;
  u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return u.v;
}

__device__ __forceinline__ f16x8 weights_f16(uint32_t w) {
  union {
    f16x2 h[4];
    f16x8 v;
  } u;
  u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0);
  u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
  u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2);
  u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
  return u.v;
}

// Eight f32 values as three bf16 vectors whose sum is exact (bits below 2^-133
// aside): each part is the top 16 bits of what the parts before it left.  Infinities and NaN stay
// in the first part (inf - inf would make them NaN).
__device__ __forceinline__ void split_f32(const u32x4 &p, const u32x4 &q, bf16x8 &hi, bf16x8 &mid, bf16x8 &lo) {
  const uint32_t v[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
  uint32_t h[8], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // a NaN whose payload sits in the low half keeps its quiet bit
    const bool special = (v[i] & 0x7F800000u) == 0x7F800000u;
    const uint32_t keep = special && (v[i] & 0x007FFFFFu) ? 0x00400000u : 0u;
    h[i] = v[i] | keep;
    const float r = special ? 0.0f : __uint_as_float(v[i]) - __uint_as_float(v[i] & 0xFFFF0000u);
    m[i] = __float_as_uint(r);
    l[i] = __float_as_uint(r - __uint_as_float(m[i] & 0xFFFF0000u));
  }
  union {
    uint32_t u[4];
    bf16x8 v;
  } a, b, c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a.u[i] = (h[2 * i] >> 16) | (h[2 * i + 1] & 0xFFFF0000u);
    b.u[i] = (m[2 * i] >> 16) | (m[2 * i + 1] & 0xFFFF0000u);
    c.u[i] = (l[2 * i] >> 16) | (l[2 * i + 1] & 0xFFFF0000u);
  }
  hi = a.v;
  mid = b.v;
  lo = c.v;
}

}  // namespace

// Workgroup: 16 rows (or, with ids, one row) x 16*NT columns, all of K;
// wave w takes steps w, w + WK, ... with D steps in flight.  With `gated`
// the first NT/2 subtiles are gate columns and the others their up columns.
template <int XT, int NT, int WK, int D>
__global__ __launch_bounds__(64 * WK) void gemv_kernel(const GemvArgs a, int first_tile) {
  constexpr int XL = XT == kF32 ? 8 : 4;  // 16-byte loads of x per step
  constexpr int ES = XT == kF32 ? 4 : 2;  // bytes per element of x
  constexpr int NSD = NT > 1 ? NT : 1;
  __shared__ __attribute__((aligned(16))) float red[WK * NT * 256];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, q4 = lane >> 4;
  const int N = a.N, K = a.K;
  const int KS = (K + 127) >> 7;
  const int G = K >> 5;
  const int gp = (G + 7) & ~7;

  const int row_tile = first_tile + blockIdx.y;
  int row0 = row_tile * 16, rows = a.M - row0;
  int64_t xrow = row0;
  const uint8_t *Bw = a.Bw, *Bs = a.Bs;
  const int out_cols = a.gated ? N >> 1 : N;
  const int cols = a.gated ? 8 * NT : 16 * NT;  // output columns of this workgroup
  const int b_bytes = (N >> 4) * K * 8;
  const int s_bytes = ((N + 255) >> 8) * 8 * gp * 32;
  bool live = true;
  if (a.ids) {
    row0 = row_tile;
    rows = 1;
    xrow = row0 / a.repeat;
    const int id = __builtin_amdgcn_readfirstlane(a.ids[row0]);
    live = id >= 0 && id < a.experts;
    const int64_t e = live ? id : 0;
    Bw += e * b_bytes;
    Bs += e * s_bytes;
  }
  if (rows > 16) rows = 16;

  const uint8_t *x = (const uint8_t *)a.x + xrow * a.ldx * ES;
  const int ldx = (int)a.ldx * ES;
  const int x_bytes = (rows - 1) * ldx + K * ES;
  const __amdgpu_buffer_rsrc_t x_rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)x, 0, x_bytes, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t b_rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)Bw, 0, b_bytes, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t s_rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)Bs, 0, s_bytes, kRsrcWord3);

  // 16-row groups of B this workgroup reads; groups past N (the last
  // workgroup of an N that is no multiple of the tile) load zeros
  const int groups = N >> 4;
  const int first = blockIdx.x * (cols >> 4);
  int gw[NT];
  bool gok[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (a.gated) {
      const int c = first + (nt % (NT > 1 ? NT / 2 : 1));
      gok[nt] = c < (groups >> 1);
      gw[nt] = nt < NT / 2 ? c : (groups >> 1) + c;
    } else {
      gw[nt] = first + nt;
      gok[nt] = gw[nt] < groups;
    }
  }

  struct Stage {
    u32x4 x[XL];
    u32x4 b[NT];
    uint32_t s[NSD];
  };
  const int steps = live ? KS : 0;
  auto load = [&](int ks, Stage &st) {
    const bool ok = ks < steps;
    const bool bk = ok && 4 * ks + q4 < G;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      st.b[nt] = __builtin_amdgcn_raw_buffer_load_b128(
          b_rsrc, off_or_oob(bk && gok[nt], gw[nt] * K * 8 + ks * 1024 + lane * 16), 0, 0);
      st.s[nt] = __builtin_amdgcn_raw_buffer_load_b32(
          s_rsrc, off_or_oob(ok && gok[nt], (gw[nt] >> 1) * gp * 32 + (ks >> 1) * 256 + lane * 4), 0, 0);
    }
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      // first element of the 16 bytes, in the order the products take them
      const int el = XT == kF16 ? i * 32 + q4 * 8 : q4 * 32 + i * (16 / ES);
      const int g = 4 * ks + (XT == kF16 ? i : q4);
      st.x[i] = __builtin_amdgcn_raw_buffer_load_b128(
          x_rsrc, off_or_oob(ok && n16 < rows && g < G, n16 * ldx + (ks * 128 + el) * ES), 0, 0);
    }
  };

  v4f acc[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) acc[nt] = v4f{0.f, 0.f, 0.f, 0.f};

  // bf16 and f32 rows: bf16 does not hold every weight of a scale beyond
  // kLargestScale.  The steps note the largest scale; where it is beyond, which
  // no model's weights are, the sums start again with kLargestScale in its
  // place: all groups (pass 0), and such a one again (pass 1, and 2 and 3) until
  // its 2 or 4 times are together.
  uint32_t largest = 0;
  auto compute = [&](int ks, const Stage &st, auto again, int pass) {
    bf16x8 part[XT == kF32 ? 3 : 1][4];
    if constexpr (XT == kF32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) split_f32(st.x[2 * i], st.x[2 * i + 1], part[0][i], part[1][i], part[2][i]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // byte (row block half) + 2 * (step parity) of the scale dword
      const uint32_t sbits = ((st.s[nt] >> (8 * ((gw[nt] & 1) + 2 * (ks & 1)))) & 0xFFu) << 23;
      if constexpr (XT == kF16) {
        uint32_t d0 = st.b[nt].x, d1 = st.b[nt].y, d2 = st.b[nt].z, d3 = st.b[nt].w;
        swap32(d0, d2);
        swap32(d1, d3);
        swap16(d0, d1);
        swap16(d2, d3);
        // the four groups' scales, each in every lane of its column
        uint32_t s0 = sbits, s2 = sbits;
        swap32(s0, s2);
        uint32_t s1 = s0, s3 = s2;
        swap16(s0, s1);
        swap16(s2, s3);
        const uint32_t d[4] = {d0, d1, d2, d3};
        const uint32_t s[4] = {s0, s1, s2, s3};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f16x8 w = weights_f16(d[i]);
          // scale byte 0 stands for 2^-127
          const float sc = s[i] ? __uint_as_float(s[i]) : __uint_as_float(0x00400000u);
          const v4f p = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, st.x[i]), w,
                                                               v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[nt][r] += p[r] * sc;
        }
      } else {
        uint32_t d[4] = {st.b[nt].x, st.b[nt].y, st.b[nt].z, st.b[nt].w};
        uint32_t scale = sbits;
        if constexpr (decltype(again)::value) {
          const int times = sbits > kLargestScale ? 1 << ((sbits - kLargestScale) >> 23) : 1;
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = times > pass ? d[i] : 0;
          scale = sbits < kLargestScale ? sbits : kLargestScale;
          // the four lanes of a column hold four of its groups, and of its sums
          if ((__ballot(sbits == kNanScale) >> n16) & 0x0001000100010001ull)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[nt][r] = __builtin_nanf("");
        } else {
          largest = sbits > largest ? sbits : largest;
        }
        const float sc = __uint_as_float(scale);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8 w = weights_bf16(d[i], sc);
          if constexpr (XT == kF32) {
#pragma unroll
            for (int h = 2; h >= 0; --h)
              acc[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(part[h][i], w, acc[nt], 0, 0, 0);
          } else {
            acc[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, st.x[i]), w, acc[nt], 0, 0, 0);
          }
        }
      }
    }
  };

  // Steps past K load zeros and add nothing, so the loop has no branch
  // between a load and its use.  The last round loads nothing: out-of-range
  // loads cost the address unit as much as others (one more round of them made
  // one row of 4096 x 512 4.2 us instead of 3.5).
  Stage st[D];
#pragma unroll
  for (int d = 0; d < D; ++d) load(wave + WK * d, st[d]);
  const int rounds = (KS + WK * D - 1) / (WK * D);
  for (int it = 0; it + 1 < rounds; ++it) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      compute(wave + WK * (it * D + d), st[d], std::false_type{}, 0);
      load(wave + WK * ((it + 1) * D + d), st[d]);
    }
  }
#pragma unroll
  for (int d = 0; d < D; ++d) compute(wave + WK * ((rounds - 1) * D + d), st[d], std::false_type{}, 0);
  if constexpr (XT != kF16) {
    if (__builtin_expect(__ballot(largest > kLargestScale) != 0, 0)) {
      const int passes = __ballot(largest >= 254u << 23) ? 4 : 2;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[nt] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int pass = 0; pass < passes; ++pass)
#pragma unroll 1
        for (int ks = wave; ks < steps; ks += WK) {
          load(ks, st[0]);
          compute(ks, st[0], std::true_type{}, pass);
        }
    }
  }

#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (4 * q4 + r < rows) red[(wave * NT + nt) * 256 + r * 64 + lane] = acc[nt][r];
  __syncthreads();
  auto sum = [&](int row, int nt, int n) {
    const int at = nt * 256 + (row & 3) * 64 + (row >> 2) * 16 + n;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) v += red[w * NT * 256 + at];
    return v;
  };
  const int shift = a.gated ? kLog2<8 * NT> : kLog2<16 * NT>;  // of cols
  for (int j = threadIdx.x; j < rows << shift; j += 64 * WK) {
    const int row = j >> shift, c = j - (row << shift);
    const int col = blockIdx.x * cols + c;
    if (col >= out_cols) continue;
    float v = sum(row, c >> 4, c & 15);
    if (a.gated) v = gated_silu(v, sum(row, NT / 2 + (c >> 4), c & 15));
    store_as(a.y, a.y_type, (size_t)(row0 + row) * a.ldy + col, v);
  }
}

constexpr int kMaxGridY = 65535;

template <int XT, int NT, int WK, int D>
static hipError_t run_gemv(const GemvArgs &a, hipStream_t stream) {
  const int cols = a.gated ? 8 * NT : 16 * NT;
  const int out_cols = a.gated ? a.N >> 1 : a.N;
  const int tiles = a.ids ? a.M : (a.M + 15) / 16;
  for (int first = 0; first < tiles; first += kMaxGridY) {
    const dim3 grid((out_cols + cols - 1) / cols, tiles - first < kMaxGridY ? tiles - first : kMaxGridY);
    gemv_kernel<XT, NT, WK, D><<<grid, 64 * WK, 0, stream>>>(a, first);
  }
  return hipGetLastError();
}

// The times below are those of calls in a graph over weights not read before.
// 16 rows a workgroup whatever M is: reading B again for the next 16, from L2,
// cost no more than tiles of 32 or 64 rows with their fewer workgroups (256
// rows of 4096 x 4096, bf16: 23.5 us, 22.5 and 23.7), and less for few rows.
// Column tiles by how many workgroups they leave: 64 columns where that makes
// one a CU or more (32 expert rows of 4096 x 2048 24.7 against 26.1 us with 32
// columns, 64 rows of 7168 x 2048 9.1 against 11.6), 16 where 32 would leave
// half the CUs idle (13 rows of 2112 x 7168 8.4 against 9.6 us), 32 otherwise
// (one row of 7168 x 7168 7.0 us; 64 columns 8.5, 16 7.7).  Four waves where
// that leaves none without a step.  One step a wave and round: two in flight
// were slower on all of these.
template <int XT>
static hipError_t run_gemv_rows(const GemvArgs &a, hipStream_t stream) {
  const int64_t row_tiles = a.ids ? a.M : (a.M + 15) / 16;
  if (row_tiles * (a.N / 64) >= 256) return run_gemv<XT, 4, 4, 1>(a, stream);
  if (a.gated || row_tiles * (a.N / 32) >= 128)
    return a.K <= 4 * 128 ? run_gemv<XT, 2, 4, 1>(a, stream) : run_gemv<XT, 2, 8, 1>(a, stream);
  return run_gemv<XT, 1, 8, 1>(a, stream);
}

hipError_t launch_gemv(const GemvArgs &a, hipStream_t stream) {
  if (a.x_type == kF16) return run_gemv_rows<kF16>(a, stream);
  if (a.x_type == kF32) return run_gemv_rows<kF32>(a, stream);
  return run_gemv_rows<kBf16>(a, stream);
}

}  // namespace mxfp4
