// The MXFP4 product of ragged row groups, one weight matrix per group:
//   C[p] = Q(A[row(p)]) * B_e^T   for offsets[e] <= p < offsets[e + 1]
// with row(p) = rows[p] / repeat, or p without `rows`; and its gated form.
//
// Two launches.  The first gathers the rows of each group, quantizes them and
// writes them in the layout that the matrix instruction takes, so that the
// second reads every operand as whole 1 KiB blocks.  The group sizes stay on
// the device: the first launch finds its rows from the offsets by a scan over
// the experts and lists the units of work for the second; grids are sized for
// the worst case.
#include "grouped_device.hpp"
#include "grouped_tile.hpp"

namespace mxfp4 {

namespace {

int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

// Units of `rows` rows that R rows in E groups can make at most: every group
// wastes less than one, and no more groups have rows than there are rows.
int64_t most_units(int64_t R, int64_t E, int64_t rows) { return (R + (rows - 1) * least(E, R)) / rows; }

int64_t k_steps(int64_t K) { return (K + 127) / 128; }

// Workspace: the list of units (16 rows each at most), codes, scales.
int64_t plan_bytes(int64_t R, int64_t E) { return (16 * (1 + most_units(R, E, 16)) + 255) / 256 * 256; }

}  // namespace

size_t grouped_workspace_bytes(int64_t R, int64_t K, int64_t E) {
  return (size_t)(plan_bytes(R, E) + most_units(R, E, 64) * k_steps(K) * (4096 + 256));
}

// Cache policy of a buffer load: the line is the first to go.
constexpr int kNonTemporal = 2;

// Gather and quantize.  One wave takes one K step of a quad, the four waves of
// a workgroup four consecutive ones, and workgroups next to each other the
// steps of one quad, so that rows are read in long runs.  Four lanes share a
// group of 32 elements (as in the large-M product's quantizer), so a load
// covers 16 rows of 64 bytes; all 16 loads of a wave are issued before the
// first is used.  Rows past the group and groups past K load as zeros and
// become zero codes with scale byte 0.  Reading the rows bounds it: 32768 rows of
// 2048 take 39 us (171 MB, 4.3 TB/s), gathered from 4096 tokens 23 us.
__global__ __launch_bounds__(256) void pack_rows_kernel(const GroupedArgs a, int runs) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int KS = (a.K + 127) >> 7;
  const GroupScan groups(a, lane);
  const int quad = blockIdx.x / runs;  // of `runs` workgroups each
  const int run = blockIdx.x - quad * runs;

  // the first workgroup past the quads lists the units
  if (quad == a.quads) {
    if (run == 0 && wave == 0) groups.list(a, lane);
    return;
  }

  // output rows of no group are zero
  if (run == 0) {
    int lo, hi, unused;
    group_range(a, 0, lo, unused);
    group_range(a, a.E - 1, unused, hi);
    const int cols = a.gated ? a.N >> 1 : a.N;
    const int outside = lo + (a.R - hi);
    for (int i = quad; i < outside; i += a.quads) {
      uint16_t *c = a.C + (int64_t)(i < lo ? i : hi + i - lo) * a.ldc;
      for (int n = threadIdx.x; n < cols; n += 256) c[n] = 0;
    }
  }

  if (quad >= groups.quads) return;
  const Unit u = groups.quad(a, quad);
  const int ks = run * 4 + wave;
  if (u.expert < 0 || ks >= KS) return;

  // the row of A of each of the quad's rows, one a lane
  int from = -1;
  if (lane < u.rows) {
    const int p = u.row + lane;
    from = a.rows ? a.rows[p] : p;
    if (a.rows) from = from < 0 ? -1 : from / a.repeat;
    if (from >= a.a_rows) from = -1;
  }
  u32x4 w[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int src = __shfl(from, 16 * j + (lane >> 2));
    const bool ok = src >= 0;
    const uint16_t *row = a.A + (int64_t)(ok ? src : 0) * a.lda;
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
      const int k = ks * 128 + ch * 32 + (lane & 3) * 8;
      w[j][ch] = u32x4{0, 0, 0, 0};
      if (ok && k < a.K) w[j][ch] = *(const u32x4 *)(row + k);
    }
  }
  const int live = (u.rows + 15) >> 4;  // tiles with a row
  uint32_t *codes = (uint32_t *)(a.codes + ((int64_t)u.tile * KS + ks) * 1024);
  uint32_t dw[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j < live) {
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t s;
        // lane = 4 * row + quarter: dword (16 * ch + row) * 4 + quarter of the block
        codes[(int64_t)j * KS * 256 + ch * 64 + lane] = quant_quarter(w[j][ch], a.sw, &s);
        dw[ch] |= s << (8 * j);
      }
    }
  }
  // lane 4 * row + c writes the scales of operand lane 16 * c + row
  const int c = lane & 3;
  uint32_t d;
  if (a.pairs) {
    // chunks c / 2 and c / 2 + 2 of blocks c % 2 and c % 2 + 2
    const uint32_t first = (c & 2 ? dw[1] : dw[0]) >> (8 * (c & 1)), second = (c & 2 ? dw[3] : dw[2]) >> (8 * (c & 1));
    d = (first & 0xFF) | ((second & 0xFF) << 8) | (first & 0xFF0000) | ((second & 0xFF0000) << 8);
  } else {
    d = c == 0 ? dw[0] : (c == 1 ? dw[1] : (c == 2 ? dw[2] : dw[3]));
  }
  ((uint32_t *)(a.scales + ((int64_t)(u.tile >> 2) * KS + ks) * 256))[c * 16 + (lane >> 2)] = d;
}

// Few rows a group, or few columns: 16 rows of one group x 16 * NT columns a
// workgroup, all of K.  Reading the weights bounds it, so operands go straight
// to registers and nothing waits at a barrier before the sums; the WK waves
// take every WK-th K step and add their tiles through LDS in wave order.  With
// `gated` the first NT / 2 subtiles are gate columns and the others their up
// columns.  Units of 16 rows also where groups hold more: 64-row units read
// the weights once instead of up to four times, but from L2 those repeats cost
// less than the workgroups they spare (771 rows of 16 experts, 2112 x 704: 10.0
// us with 64 rows, 8.4 with 16).  256 rows of 64 experts, 4096 x 2048: 42 to 45 us
// by the run, 6.2 TB/s of weights and more.  With the weights through the caches,
// then 46.8 us: 32 columns or 8 waves instead 48.9 and 46.4, but 17.2 and 17.5 for
// 15.2 of 700 rows of 32 experts, 4096 x 1024.
// ONCE: weights that no cache will hold until they are read again go past them.
template <int NT, int WK, bool ONCE>
__global__ __launch_bounds__(64 * WK) void grouped_stream_kernel(const GroupedArgs a, int n_tiles) {
  __shared__ __attribute__((aligned(16))) float red[WK * NT * 256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q4 = lane >> 4;
  const int N = a.N, K = a.K;
  const int KS = (K + 127) >> 7;
  const int gp = ((K >> 5) + 7) & ~7;
  const int b_bytes = (N >> 4) * K * 8;
  const int s_bytes = ((N + 255) >> 8) * 8 * gp * 32;
  const int groups = N >> 4;
  const int out_cols = a.gated ? N >> 1 : N;
  const int shift = a.gated ? kLog2<8 * NT> : kLog2<16 * NT>;  // of the columns of a tile

  const int64_t work = (int64_t)unit_count(a) * n_tiles;
  for (int64_t item = blockIdx.x; item < work; item += gridDim.x) {
    const int index = (int)(item / n_tiles);
    const int n_tile = (int)(item - (int64_t)index * n_tiles);
    const Unit u = plan_entry<16>(a, 1 + index);
    if (u.expert < 0) continue;

    const int rows = u.rows < 16 ? u.rows : 16;
    const __amdgpu_buffer_rsrc_t a_rsrc =
        __builtin_amdgcn_make_buffer_rsrc((void *)(a.codes + (int64_t)u.tile * KS * 1024), 0, KS * 1024, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t as_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(a.scales + (int64_t)(u.tile >> 2) * KS * 256), 0, KS * 256, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t b_rsrc =
        __builtin_amdgcn_make_buffer_rsrc((void *)(a.Bw + (int64_t)u.expert * b_bytes), 0, b_bytes, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t s_rsrc =
        __builtin_amdgcn_make_buffer_rsrc((void *)(a.Bs + (int64_t)u.expert * s_bytes), 0, s_bytes, kRsrcWord3);
    const int first = n_tile << (shift - 4);
    int gw[NT];
    bool gok[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (a.gated) {
        const int c = first + (nt % (NT / 2));
        gok[nt] = c < (groups >> 1);
        gw[nt] = nt < NT / 2 ? c : (groups >> 1) + c;
      } else {
        gw[nt] = first + nt;
        gok[nt] = gw[nt] < groups;
      }
    }
    const int tile_shift = 8 * (u.tile & 3);  // of the rows' byte in a scale dword

    struct Stage {
      u32x4 x;
      uint32_t xs;
      u32x4 b[NT];
      uint32_t s[NT];
    } st;
    auto load = [&](int ks) {
      const bool ok = ks < KS;
      // a K chunk past the end meets zeros of the rows; it must not run past
      // the matrix all the same
      const bool bk = ok && (4 * ks + q4) * 32 < K;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        st.b[nt] = __builtin_amdgcn_raw_buffer_load_b128(
            b_rsrc, off_or_oob(bk && gok[nt], gw[nt] * K * 8 + ks * 1024 + lane * 16), 0, ONCE ? kNonTemporal : 0);
        st.s[nt] = __builtin_amdgcn_raw_buffer_load_b32(
            s_rsrc, off_or_oob(ok && gok[nt], (gw[nt] >> 1) * gp * 32 + (ks >> 1) * 256 + lane * 4), 0, 0);
      }
      st.x = __builtin_amdgcn_raw_buffer_load_b128(a_rsrc, off_or_oob(ok, ks * 1024 + lane * 16), 0, 0);
      st.xs = __builtin_amdgcn_raw_buffer_load_b32(as_rsrc, off_or_oob(ok, ks * 256 + lane * 4), 0, 0);
    };
    v4f acc[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[nt] = v4f{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](int ks) {
      const uint32_t sa = (st.xs >> tile_shift) & 0xFFu;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t sb = (st.s[nt] >> (8 * ((gw[nt] & 1) + 2 * (ks & 1)))) & 0xFFu;
        acc[nt] = mfma_fp4(st.x, st.b[nt], acc[nt], sa, sb);
      }
    };
    // Steps past K load zeros and add nothing; the last round loads nothing.
    const int rounds = (KS + WK - 1) / WK;
    load(wave);
    for (int it = 0; it + 1 < rounds; ++it) {
      compute(wave + WK * it);
      load(wave + WK * (it + 1));
    }
    compute(wave + WK * (rounds - 1));

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[(wave * NT + nt) * 256 + r * 64 + lane] = acc[nt][r];
    __syncthreads();
    auto sum = [&](int row, int nt, int n) {
      const int at = nt * 256 + (row & 3) * 64 + (row >> 2) * 16 + n;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < WK; ++w) v += red[w * NT * 256 + at];
      return v;
    };
    for (int j = threadIdx.x; j < rows << shift; j += 64 * WK) {
      const int row = j >> shift, c = j - (row << shift);
      const int col = (n_tile << shift) + c;
      if (col >= out_cols) continue;
      float v = sum(row, c >> 4, c & 15);
      if (a.gated) v = gated_silu(v, sum(row, NT / 2 + (c >> 4), c & 15));
      ((__bf16 *)a.C)[(int64_t)(u.row + row) * a.ldc + col] = (__bf16)v;
    }
    __syncthreads();  // before the next item's sums
  }
}

// Workgroups of a launch (threads of a grid dimension are limited to 2^32).
constexpr int64_t kMaxGrid = 1 << 22;

// Whether the weights go past the caches: 8 rows a group at most on average, so
// that few groups have a second unit, and matrices of 96 MiB or more in all,
// which the caches do not keep until a later call wants the same ones, beside
// everything else.  It goes by all of them, also where there are fewer rows than
// groups.  Both launches, 4096 x 2048 gated (4 MiB of codes a matrix), weights that
// other calls' have displaced, through the caches and past them: 64 experts with
// a row each 53.6 and 49.8 us, 4 rows 54.4 and 50.6, 8 rows 55.6 and 51.9, 16 rows
// 57.8 and 61.2; 512 rows of which one expert has 449 64.5 and 63.8; 8 rows of 8 of
// them 12.5 and 11.9, 23 of 23 24.2 and 22.7.  Where nothing came in between, 64
// groups of 4 rows 48.5 and 50.2, 512 rows with one of 449 58.9 and 63.9, 8 rows
// 10.7 to 11.5 and 10.4 to 11.7 by the run.
static bool read_once(const GroupedArgs &a) {
  return a.R / least(a.E, a.R) <= 8 && (int64_t)a.E * a.N * (a.K / 2) >= (int64_t)96 << 20;
}

static hipError_t run_stream(const GroupedArgs &a, hipStream_t stream) {
  const int cols = a.gated ? 32 : 64;
  const int out_cols = a.gated ? a.N >> 1 : a.N;
  const int n_tiles = (out_cols + cols - 1) / cols;
  const int64_t items = (int64_t)a.max_units * n_tiles;
  const unsigned grid = (unsigned)least(items, kMaxGrid);
  if (read_once(a))
    grouped_stream_kernel<4, 4, true><<<grid, 256, 0, stream>>>(a, n_tiles);
  else
    grouped_stream_kernel<4, 4, false><<<grid, 256, 0, stream>>>(a, n_tiles);
  return hipGetLastError();
}

static int tile_columns(const GroupedArgs &a) { return a.gated ? (a.N / 2 + 127) / 128 : (a.N + 255) / 256; }

static hipError_t run_tile(const GroupedArgs &a, hipStream_t stream) {
  const int wide = ((uintptr_t)a.C & 15) == 0 && a.ldc % 8 == 0;
  if (a.gated)
    grouped_tile_kernel<true><<<512, 256, 0, stream>>>(a, tile_columns(a), wide);
  else
    grouped_tile_kernel<false><<<512, 256, 0, stream>>>(a, tile_columns(a), wide);
  return hipGetLastError();
}

// Whether the 128-row tiles are the faster form: groups of 32 rows on average
// and a tile for every CU.  Both timed on groups of one size, 16-row units
// against tiles: 2048 rows of 64 experts, 2048 x 1024: 18.5 and 16.9 us; 4096
// rows, 4096 x 2048: 98 and 72.  Below either bound: 1280 rows (20 a group) of 4096
// x 1024 31.8 and 34.5; 256 rows of 8 experts, 4096 x 2048 (128 tiles) 9.9 and
// 12.1.  The tiles also need their pairs of column groups whole.
static bool use_tiles(const GroupedArgs &a) {
  const int64_t some = least(a.E, a.R);
  const int64_t units = a.R / 128 > some ? a.R / 128 : some;
  return a.R / some >= 32 && units * tile_columns(a) >= 256 && a.N % (a.gated ? 64 : 32) == 0;
}

hipError_t launch_grouped(GroupedArgs a, hipStream_t stream) {
  const int64_t quads = most_units(a.R, a.E, 64), KS = k_steps(a.K);
  const bool tiles = use_tiles(a);
  a.pairs = tiles;
  a.unit_shift = tiles ? 7 : 4;
  a.unit_rows = 1 << a.unit_shift;
  a.max_units = (int)most_units(a.R, a.E, a.unit_rows);
  a.quads = (int)quads;
  a.plan = (int4 *)a.ws;
  a.codes = a.ws + plan_bytes(a.R, a.E);
  a.scales = a.codes + quads * KS * 4096;
  const int64_t runs = (KS + 3) / 4;
  pack_rows_kernel<<<(unsigned)(quads * runs + 1), 256, 0, stream>>>(a, (int)runs);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return tiles ? run_tile(a, stream) : run_stream(a, stream);
}

}  // namespace mxfp4
