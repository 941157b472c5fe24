// The dense layer on MXFP4 weights:
//   z = Q(x) * B^T + bias,  y = f(z) + residual,
// or, gated, y = f(first half of z's columns) * second half + residual.
//
// More than a few rows are quantized into the prepared layout by a launch of
// their own, so that both operands of the product are read as whole blocks; a
// few are quantized by the product's waves themselves (in_one_launch).
#include "linear_bounds.hpp"
#include "linear_epilogue.hpp"
#include "linear_internal.hpp"

namespace mxfp4 {

// Quantize rows into the prepared layout.  One wave takes one K step of 16
// rows, as prepare_b does; four lanes share a group of 32 elements.  Rows past
// the last one and groups past K become zero codes; where the last 16 rows are
// the first of their block of 32, the scale bytes of the others are zero too.
// Bytes bound it: 8192 rows of 8192, 170 MB, in 29 us, 5.9 TB/s.
template <bool SW>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const uint16_t *x, int64_t ld, int rows, int K, uint8_t *codes,
                                                        uint8_t *scales, int steps, int units) {
  const int lane = threadIdx.x & 63;
  const int unit = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= units) return;
  const int g = unit / steps, s = unit - g * steps;
  const int G = K >> 5, gp = (G + 7) & ~7;
  const int row = 16 * g + (lane >> 2);
  const bool live = row < rows;
  const uint16_t *from = x + (int64_t)(live ? row : 0) * ld + (lane & 3) * 8;
  u32x4 w[4];
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    w[ch] = u32x4{0, 0, 0, 0};
    if (live && 4 * s + ch < G) w[ch] = *(const u32x4 *)(from + (4 * s + ch) * 32);
  }
  uint32_t *to = (uint32_t *)(codes + (int64_t)g * K * 8);
  uint8_t *block = scales + (int64_t)(row >> 5) * 32 * gp;
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    const int grp = 4 * s + ch;
    uint32_t sc;
    const uint32_t d = quant_quarter_t<SW>(w[ch], &sc);
    if (grp < G) to[grp * 64 + lane] = d;
    if ((lane & 3) == 0 && grp < gp) {
      uint8_t *const at = block + shuffled_scale_offset(row & 31, grp, gp);
      *at = (uint8_t)sc;
      if (!(g & 1) && 16 * (g + 1) >= rows) at[1] = 0;  // row + 16
    }
  }
}

hipError_t launch_pack_rows(const uint16_t *x, int64_t ld, int64_t rows, int64_t K, uint8_t *codes, uint8_t *scales,
                            bool sw, hipStream_t stream) {
  const int steps = (int)((K / 32 + 7) / 8 * 2);  // the scales' padding included
  const int64_t units = (rows + 15) / 16 * steps;
  const unsigned blocks = (unsigned)((units + 3) / 4);
  if (sw)
    quantize_rows_kernel<true><<<blocks, 256, 0, stream>>>(x, ld, (int)rows, (int)K, codes, scales, steps, (int)units);
  else
    quantize_rows_kernel<false><<<blocks, 256, 0, stream>>>(x, ld, (int)rows, (int)K, codes, scales, steps, (int)units);
  return hipGetLastError();
}

// 16 * MW rows x 16 * NT weight rows a workgroup; the WK waves take every
// WK-th K step, D of them loaded ahead, hold the whole tile's sums and add them
// through LDS in wave order.  Nothing waits at a barrier before that.  The weights
// are the first operand of the instruction, so a lane holds four neighbouring
// columns of a row.  Gated: the first NT / 2 weight groups are gate columns, the
// others their up columns.
// PACKED: the rows come quantized.  Otherwise each wave quantizes them on its
// way: the operand's lane has 32 elements of one row, a whole group, so the
// scale is found and the codes are made without another lane's help.
// One row of 4096 x 4096: 4.0 us at least, of which a launch is 2; gated 16384 x 4096
// 6.4, reading 36 MB at 5.6 TB/s launch included.  13 rows of 2112 x 7168 8.2: each
// of 132 workgroups takes in all rows, 186 KB, beside 61 KB of weights.  D of 3 or 4
// instead of 2 and 16 waves instead of 8 were slower (a K of 4096 is 4 steps a wave of 8).
template <int MW, int NT, int WK, int D, bool PACKED>
__global__ __launch_bounds__(64 * WK) void linear_split_kernel(const LinearArgs a, int n_tiles, int first_m) {
  __shared__ __attribute__((aligned(16))) v4f red[WK][MW * NT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m_here = blockIdx.x / n_tiles, n_tile = blockIdx.x - m_here * n_tiles;
  const int m_tile = first_m + m_here;
  const int K = a.K, N = a.N;
  const int KS = (K + 127) >> 7;
  const int gp = ((K >> 5) + 7) & ~7;
  const int groups = N >> 4;
  const int row0 = m_tile * 16 * MW;
  const int x_groups = (a.M + 15) >> 4, xg0 = m_tile * MW;
  const int q4 = lane >> 4;

  const int64_t b_bytes = (int64_t)groups * K * 8, s_bytes = (int64_t)((N + 255) >> 8) * 8 * gp * 32;
  const __amdgpu_buffer_rsrc_t b_rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)a.Bw, 0, (int)b_bytes, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t s_rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)a.Bs, 0, (int)s_bytes, kRsrcWord3);
  // the rows: their codes and scales, or themselves
  const int own_groups = x_groups - xg0 < MW ? x_groups - xg0 : MW;
  const int ldx = (int)a.ldx * 2;
  const int own_rows = a.M - row0 < 16 * MW ? a.M - row0 : 16 * MW;
  const __amdgpu_buffer_rsrc_t x_rsrc =
      PACKED ? __builtin_amdgcn_make_buffer_rsrc((void *)(a.codes + (int64_t)xg0 * K * 8), 0, own_groups * K * 8, kRsrcWord3)
             : __builtin_amdgcn_make_buffer_rsrc((void *)(a.x + (int64_t)row0 * a.ldx), 0, (own_rows - 1) * ldx + K * 2,
                                                 kRsrcWord3);
  const __amdgpu_buffer_rsrc_t xs_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void *)(a.scales + (int64_t)(xg0 >> 1) * gp * 32), 0,
      PACKED ? (((xg0 & 1) + own_groups + 1) >> 1) * gp * 32 : 0, kRsrcWord3);

  int gw[NT];
  bool gok[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (a.gated) {
      const int c = n_tile * (NT / 2) + nt % (NT > 1 ? NT / 2 : 1);
      gok[nt] = c < (groups >> 1);
      gw[nt] = nt < NT / 2 ? c : (groups >> 1) + c;
    } else {
      gw[nt] = n_tile * NT + nt;
      gok[nt] = gw[nt] < groups;
    }
    gw[nt] = group_within(gw[nt], groups);
  }
  v4f acc[MW][NT];
#pragma unroll
  for (int mt = 0; mt < MW; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = v4f{0.f, 0.f, 0.f, 0.f};

  struct Stage {
    u32x4 x[MW][PACKED ? 1 : 4], b[NT];
    uint32_t xs[MW], bs[NT];
  } st[D];
  auto load = [&](int q, int ks) __attribute__((always_inline)) {
    // a K chunk past the end meets zeros of the rows; it must not run past
    // the matrix all the same (its offset may pass 2^31, hence unsigned)
    const bool ok = (4 * ks + q4) * 32 < K;
    if (!PACKED)
#pragma unroll
      for (int mt = 0; mt < MW; ++mt) {
        const int row = 16 * mt + (lane & 15);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st[q].x[mt][i] = __builtin_amdgcn_raw_buffer_load_b128(
              x_rsrc, off_or_oob(ok && row < own_rows, row * ldx + ks * 256 + q4 * 64 + 16 * i), 0, 0);
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      st[q].b[nt] = __builtin_amdgcn_raw_buffer_load_b128(
          b_rsrc, off_or_oob(ok && gok[nt], (int)((uint32_t)(gw[nt] * K * 8) + ks * 1024 + lane * 16)), 0, 0);
      st[q].bs[nt] = __builtin_amdgcn_raw_buffer_load_b32(
          s_rsrc, off_or_oob(ok && gok[nt], (gw[nt] >> 1) * gp * 32 + (ks >> 1) * 256 + lane * 4), 0, 0);
    }
    if (PACKED)
#pragma unroll
      for (int mt = 0; mt < MW; ++mt) {
        st[q].x[mt][0] =
            __builtin_amdgcn_raw_buffer_load_b128(x_rsrc, off_or_oob(ok, mt * K * 8 + ks * 1024 + lane * 16), 0, 0);
        st[q].xs[mt] = __builtin_amdgcn_raw_buffer_load_b32(
            xs_rsrc, off_or_oob(ok, (((xg0 & 1) + mt) >> 1) * gp * 32 + (ks >> 1) * 256 + lane * 4), 0, 0);
      }
  };
  auto compute = [&](int q, int ks) __attribute__((always_inline)) {
    u32x4 x[MW];
    uint32_t xs[MW];
#pragma unroll
    for (int mt = 0; mt < MW; ++mt) {
      if (PACKED) {
        x[mt] = st[q].x[mt][0];
        xs[mt] = st[q].xs[mt] >> (8 * (((xg0 + mt) & 1) + 2 * (ks & 1)));
      } else {
        uint32_t w[16], c[4];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = st[q].x[mt][PACKED ? 0 : i >> 2][i & 3];
        xs[mt] = a.sw ? quant_group32<true>(w, c) : quant_group32<false>(w, c);
        x[mt] = u32x4{c[0], c[1], c[2], c[3]};
      }
    }
#pragma unroll
    for (int mt = 0; mt < MW; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        acc[mt][nt] = mfma_fp4(st[q].b[nt], x[mt], acc[mt][nt], st[q].bs[nt] >> (8 * ((gw[nt] & 1) + 2 * (ks & 1))), xs[mt]);
  };
#pragma unroll
  for (int q = 0; q < D; ++q) load(q, wave + q * WK);
  // steps past the last are zeros; the last round loads nothing
  int ks = wave;
  for (; ks - wave + D * WK < KS; ks += D * WK)
#pragma unroll
    for (int q = 0; q < D; ++q) {
      compute(q, ks + q * WK);
      load(q, ks + (D + q) * WK);
    }
#pragma unroll
  for (int q = 0; q < D; ++q) compute(q, ks + q * WK);
#pragma unroll
  for (int mt = 0; mt < MW; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) red[wave][mt * NT + nt][lane] = acc[mt][nt];
  __syncthreads();

  const auto sum = [&](int block, int l) {
    v4f v = red[0][block][l];
#pragma unroll
    for (int w = 1; w < WK; ++w) v += red[w][block][l];
    return v;
  };
  const int blocks = a.gated ? MW * NT / 2 : MW * NT;
  for (int j = threadIdx.x; j < blocks * 64; j += 64 * WK) {
    const int l = j & 63, block = j >> 6;
    const int across = a.gated ? NT / 2 : NT;
    const int mt = block / across, nt = block - mt * across;
    const int row = row0 + mt * 16 + (l & 15);
    const int col = (n_tile * across + nt) * 16 + (l >> 4) * 4;
    if (row >= a.M || col >= (a.gated ? N >> 1 : N)) continue;
    const v4f z = sum(mt * NT + nt, l);
    const v4f up = a.gated ? sum(mt * NT + nt + NT / 2, l) : z;
    linear_emit(a, row, col, z, up);
  }
}

// Whether 256 x 256 tiles are the faster form: one for half of the CUs.  us a call
// with them and without, rows of 4096 x 4096: 1536 (96 tiles) 39.3 and 37.5, 2048 (128)
// 40.3 and 45.2; 4096 x 1024: 20.4 and 20.9, 20.7 and 26.5; 2048 x 2048, 2560 rows (80)
// 28.6 and 27.1, 4096 (128) 30.9 and 35.8; 16384 x 4096, 264 rows (128) 40.6 and 35.0,
// 384 (128) 40.7 and 41.5, 512 (128) 41.5 and 51.  Few rows of very many columns leave
// the tiles almost empty (tiles_filled).  Gated ones need their pairs of column
// groups whole.  (Of matrices within 4 KiB of 2^31 bytes their steps past K would
// pass that.)
static bool use_tiles(const LinearArgs &a) {
  const int64_t m_tiles = (a.M + 255) / 256, n_tiles = ((int64_t)a.N + 255) / 256;
  return m_tiles * n_tiles >= 128 && tiles_filled(a.M, a.N) && (!a.gated || a.N % 64 == 0) &&
         tile_offsets_fit(a.N, a.K);
}

// Whether the rows are quantized on the way, in one launch: 16 of them at most,
// and as every workgroup reads all of them, 192 KiB.  us so and with a launch of
// their own, captured and not: 16 rows of 4096 x 4096 6.8 and 7.1, 7.9 and 11; 2112 x
// 7168, 2 rows 6.2 and 7.9, 7.5 and 11, 8 rows 7.9 and 7.8, 7.8 and 11, 13 rows 8.8 and
// 7.8, 8.5 and 11, 16 rows 9.8 and 7.9, 9.5 and 11; 16384 x 4096, 16 rows 10.5 and
// 11.7, 10.3 and 11.5.  Captured calls would rather change at an M * K of 65536, others
// beyond 114688: the bound follows the others and costs captured ones 1 us at most.
static bool in_one_launch(int64_t M, int64_t K) { return M <= 16 && M * K <= 98304; }

size_t linear_workspace_bytes(int64_t M, int64_t N, int64_t K) { return in_one_launch(M, K) ? 0 : packed_bytes(M, K); }

template <int MW, int NT, int WK, int D, bool PACKED>
static void run_split(const LinearArgs &a, hipStream_t stream) {
  const int cols = a.gated ? a.N / 2 : a.N, width = a.gated ? 8 * NT : 16 * NT;
  const int64_t n_tiles = (cols + width - 1) / width;
  const int m_tiles = (a.M + 16 * MW - 1) / (16 * MW);
  // a grid dimension holds fewer than 2^32 threads
  const int most = (int)(((int64_t)1 << 31) / (64 * WK * n_tiles)) + 1;
  for (int first = 0; first < m_tiles; first += most) {
    const int here = m_tiles - first < most ? m_tiles - first : most;
    linear_split_kernel<MW, NT, WK, D, PACKED><<<(unsigned)(n_tiles * here), 64 * WK, 0, stream>>>(a, (int)n_tiles, first);
  }
}

hipError_t launch_linear(LinearArgs a, hipStream_t stream) {
  if (in_one_launch(a.M, a.K)) {
    // 16, 32 or 64 weight rows a workgroup, so that there are 256 of them at most,
    // about.  us for one row: 4096 x 4096 4.6, 6.0 (16 and 32); gated 16384 x 4096 8.6
    // and 6.9 (32 and 64).
    if (!a.gated && a.N <= 4096)
      run_split<1, 1, 8, 2, false>(a, stream);
    else if (a.N <= 8192)
      run_split<1, 2, 8, 2, false>(a, stream);
    else
      run_split<1, 4, 8, 2, false>(a, stream);
    return hipGetLastError();
  }
  a.codes = a.ws;
  a.scales = a.ws + (packed_codes_bytes(a.M, a.K) + 255) / 256 * 256;
  const hipError_t e = launch_pack_rows(a.x, a.ldx, a.M, a.K, a.codes, a.scales, a.sw, stream);
  if (e != hipSuccess) return e;
  if (use_tiles(a)) return launch_linear_tile(a, stream);
  // Small tiles make more workgroups, large ones read less: the smallest of which
  // every CU has one at most, about.  us a call with 32 x 32, 32 x 64 and 32 x 128
  // weight rows a workgroup: 32 rows of 4096 x 4096 7.0, 8.0 and 11.5; 128 rows 9.6,
  // 8.6 and 12.0; 512 rows 22.3, 19.4 and 17.5.
  const int64_t m_tiles = (a.M + 31) / 32;
  if (a.M <= 16)
    run_split<1, 2, 8, 2, true>(a, stream);
  else if (m_tiles * ((a.N + 31) / 32) <= 256)
    run_split<2, 2, 8, 2, true>(a, stream);
  else if (m_tiles * ((a.N + 63) / 64) <= 288)
    run_split<2, 4, 8, 2, true>(a, stream);
  else
    run_split<2, 8, 4, 2, true>(a, stream);
  return hipGetLastError();
}

}  // namespace mxfp4
