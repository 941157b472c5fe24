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

// Gather and quantize.  One wave takes one K step of a quad, the four waves of
// a workgroup four consecutive ones, and workgroups next to each other the
// steps of one quad, so that rows are read in long runs.  Four lanes share a
// group of 32 elements (as in the large-M product's quantizer), so a load
// covers 16 rows of 64 bytes; all 16 loads of a wave are issued before the
// first is used.  Rows past the group and groups past K load as zeros and
// become zero codes with scale byte 0.
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

// Workgroup: 16 * MT rows of one group x 16 * NT columns, all of K; wave w
// takes steps w, w + WK, ... with D steps in flight.  With `gated` the first
// NT / 2 subtiles are gate columns and the others their up columns.
template <int MT, int NT, int WK, int D>
__global__ __launch_bounds__(64 * WK) void grouped_stream_kernel(const GroupedArgs a, int n_tiles) {
  __shared__ __attribute__((aligned(16))) float red[WK * MT * NT * 256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q4 = lane >> 4;
  const int64_t work = (int64_t)plan_entry(a, 0).expert * n_tiles;
  for (int64_t item = blockIdx.x; item < work; item += gridDim.x) {
    const int index = (int)(item / n_tiles);
    const int n_tile = (int)(item - (int64_t)index * n_tiles);
    const Unit u = plan_entry(a, 1 + index);
    if (u.expert < 0) continue;

    const int N = a.N, K = a.K;
    const int KS = (K + 127) >> 7;
    const int gp = ((K >> 5) + 7) & ~7;
    const int b_bytes = (N >> 4) * K * 8;
    const int s_bytes = ((N + 255) >> 8) * 8 * gp * 32;
    const int rows = u.rows < 16 * MT ? u.rows : 16 * MT;
    const int tiles = (rows + 15) >> 4;
    const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(a.codes + (int64_t)u.tile * KS * 1024), 0, tiles * KS * 1024, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t as_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(a.scales + (int64_t)(u.tile >> 2) * KS * 256), 0, ((MT + 3) / 4) * KS * 256, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t b_rsrc =
        __builtin_amdgcn_make_buffer_rsrc((void *)(a.Bw + (int64_t)u.expert * b_bytes), 0, b_bytes, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t s_rsrc =
        __builtin_amdgcn_make_buffer_rsrc((void *)(a.Bs + (int64_t)u.expert * s_bytes), 0, s_bytes, kRsrcWord3);

    const int groups = N >> 4;
    const int cols = a.gated ? 8 * NT : 16 * NT;
    const int first = n_tile * (cols >> 4);
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
    const int tile_shift = 8 * (u.tile & 3);  // of the first tile's byte in a scale dword (0 unless MT < 4)

    struct Stage {
      u32x4 x[MT];
      uint32_t xs[(MT + 3) / 4];
      u32x4 b[NT];
      uint32_t s[NT];
    };
    auto load = [&](int ks, Stage &st) {
      const bool ok = ks < KS;
      // a K chunk past the end meets zero rows of A; it is left out of range
      // only where it would run past the matrix
      const bool bk = ok && (4 * ks + q4) * 32 < K;
  #pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        st.b[nt] = __builtin_amdgcn_raw_buffer_load_b128(
            b_rsrc, off_or_oob(bk && gok[nt], gw[nt] * K * 8 + ks * 1024 + lane * 16), 0, 0);
        st.s[nt] = __builtin_amdgcn_raw_buffer_load_b32(
            s_rsrc, off_or_oob(ok && gok[nt], (gw[nt] >> 1) * gp * 32 + (ks >> 1) * 256 + lane * 4), 0, 0);
      }
  #pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        st.x[mt] = __builtin_amdgcn_raw_buffer_load_b128(
            a_rsrc, off_or_oob(ok && mt < tiles, (mt * KS + ks) * 1024 + lane * 16), 0, 0);
  #pragma unroll
      for (int q = 0; q < (MT + 3) / 4; ++q)
        st.xs[q] = __builtin_amdgcn_raw_buffer_load_b32(as_rsrc, off_or_oob(ok, (q * KS + ks) * 256 + lane * 4), 0, 0);
    };

    v4f acc[MT][NT];
  #pragma unroll
    for (int mt = 0; mt < MT; ++mt)
  #pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = v4f{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](int ks, const Stage &st) {
  #pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t sb = (st.s[nt] >> (8 * ((gw[nt] & 1) + 2 * (ks & 1)))) & 0xFFu;
  #pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint32_t sa = (st.xs[mt >> 2] >> (tile_shift + 8 * (mt & 3))) & 0xFFu;
          acc[mt][nt] = mfma_fp4(st.x[mt], st.b[nt], acc[mt][nt], sa, sb);
        }
      }
    };

    Stage st[D];
  #pragma unroll
    for (int d = 0; d < D; ++d) load(wave + WK * d, st[d]);
    const int rounds = (KS + WK * D - 1) / (WK * D);
    for (int it = 0; it < rounds; ++it) {
  #pragma unroll
      for (int d = 0; d < D; ++d) {
        compute(wave + WK * (it * D + d), st[d]);
        load(wave + WK * ((it + 1) * D + d), st[d]);
      }
    }

  #pragma unroll
    for (int mt = 0; mt < MT; ++mt)
  #pragma unroll
      for (int nt = 0; nt < NT; ++nt)
  #pragma unroll
        for (int r = 0; r < 4; ++r) red[((wave * MT + mt) * NT + nt) * 256 + r * 64 + lane] = acc[mt][nt][r];
    __syncthreads();
    auto sum = [&](int row, int nt, int n) {
      const int at = ((row >> 4) * NT + nt) * 256 + (row & 3) * 64 + ((row >> 2) & 3) * 16 + n;
      float v = 0.f;
  #pragma unroll
      for (int w = 0; w < WK; ++w) v += red[w * MT * NT * 256 + at];
      return v;
    };
    const int out_cols = a.gated ? N >> 1 : N;
    for (int j = threadIdx.x; j < rows * cols; j += 64 * WK) {
      const int row = j / cols, c = j - row * cols;
      const int col = n_tile * cols + c;
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

template <int MT, int NT, int WK, int D>
static hipError_t run_stream(const GroupedArgs &a, hipStream_t stream) {
  const int cols = a.gated ? 8 * NT : 16 * NT;
  const int out_cols = a.gated ? a.N >> 1 : a.N;
  const int n_tiles = (out_cols + cols - 1) / cols;
  const int64_t items = (int64_t)a.max_units * n_tiles;
  grouped_stream_kernel<MT, NT, WK, D><<<(unsigned)least(items, kMaxGrid), 64 * WK, 0, stream>>>(a, n_tiles);
  return hipGetLastError();
}

static hipError_t run_tile(const GroupedArgs &a, hipStream_t stream) {
  const int wide = ((uintptr_t)a.C & 15) == 0 && a.ldc % 8 == 0;
  if (a.gated)
    grouped_tile_kernel<true, 1><<<512, 256, 0, stream>>>(a, (a.N / 2 + 127) / 128, wide);
  else
    grouped_tile_kernel<false, 1><<<512, 256, 0, stream>>>(a, (a.N + 255) / 256, wide);
  return hipGetLastError();
}

hipError_t launch_grouped(GroupedArgs a, hipStream_t stream) {
  const int64_t quads = most_units(a.R, a.E, 64), KS = k_steps(a.K);
  const int64_t mean = a.R / least(a.E, a.R);  // rows of a group, were they even
  const bool tile = mean > 64 && a.N % (a.gated ? 64 : 32) == 0;
  a.unit_shift = tile ? 7 : (mean <= 16 ? 4 : 6);
  a.pairs = tile;
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
  if (tile) return run_tile(a, stream);
  if (mean <= 16) return run_stream<1, 2, 8, 2>(a, stream);
  return run_stream<4, 4, 4, 2>(a, stream);
}

}  // namespace mxfp4
