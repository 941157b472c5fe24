// The backward pass of the dense layer's epilogue:
//   dz = dy * f'(z), or gated dz = [dy * up * f'(gate), dy * f(gate)],
//   dbias = sum over the rows of dz, unrounded.
#include "linear_device.hpp"
#include "linear_internal.hpp"

namespace mxfp4 {

namespace {

constexpr int kCols = 256;  // output columns of a workgroup: 4 a lane
constexpr int kWaves = 4;

int64_t grad_columns(const GradPreArgs &a) { return a.gated ? a.N / 2 : a.N; }

}  // namespace

// 64 lanes x 4 neighbouring columns; the four waves take every fourth row of a
// chunk, BATCH of them loaded before the first is used.  The bias' gradient is
// summed in f32 by each lane over its rows, over the waves in LDS, and over the
// chunks by a second launch, in that order.  Bytes bound it: 8192 rows, 16384
// gated, 671 MB in 127 us, 5.3 TB/s (a copy of 1 GiB: 5.2).
// BATCH: 4 where a chunk is 16 rows, so that a wave waits for memory once (771
// rows of 2112 columns); 1 where chunks are long and other waves fill the time
// (the 8192 rows: 127 us, in fours 169).
template <bool GATED, int BATCH>
__global__ __launch_bounds__(256) void grad_pre_kernel(const GradPreArgs a) {
  __shared__ __attribute__((aligned(16))) v4f red[2][kWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = a.N >> 1;
  const int cols = GATED ? half : a.N;
  const int col = blockIdx.x * kCols + lane * 4;
  const bool live = col < cols;
  const int first = blockIdx.y * a.chunk_rows;
  const int last = first + a.chunk_rows < a.M ? first + a.chunk_rows : a.M;
  v4f sum = {0.f, 0.f, 0.f, 0.f}, sum_up = {0.f, 0.f, 0.f, 0.f};
  if (live)
    for (int row0 = first + wave; row0 < last; row0 += kWaves * BATCH) {
      v4f dy[BATCH], z[BATCH], up[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int row = row0 + b * kWaves;
        if (row >= last) break;
        dy[b] = load4(a.dy, a.dy_type, (int64_t)row * a.ld_dy + col, a.wide);
        if (a.pre) z[b] = load4(a.pre, 0, (int64_t)row * a.ld_pre + col, a.wide);
        if (GATED) up[b] = load4(a.pre, 0, (int64_t)row * a.ld_pre + half + col, a.wide);
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int row = row0 + b * kWaves;
        if (row >= last) break;
        v4f dz = dy[b];
        if (a.pre) {
          v4f f, slope;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float s;
            f[i] = activate_slope(a.act, z[b][i], s);
            slope[i] = s;
          }
          dz = dz * slope;
          if (GATED) {
            dz = dz * up[b];
            const v4f dup = dy[b] * f;
            store4(a.dz, 0, (int64_t)row * a.ld_dz + half + col, dup, a.wide);
            sum_up += dup;
          }
        }
        store4(a.dz, 0, (int64_t)row * a.ld_dz + col, dz, a.wide);
        sum += dz;
      }
    }
  if (!a.dbias) return;
  red[0][wave][lane] = sum;
  red[1][wave][lane] = sum_up;
  __syncthreads();
  if (wave < (GATED ? 2 : 1) && live) {
    v4f v = red[wave][0][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += red[wave][w][lane];
    *(v4f *)(a.partial + (int64_t)blockIdx.y * a.N + wave * half + col) = v;
  }
}

// The chunks' sums: 16 columns a workgroup, 16 threads a column, each of which
// takes every 16th chunk; they meet in LDS, in order.
__global__ __launch_bounds__(256) void sum_chunks_kernel(const float *partial, int chunks, int n, float *out) {
  __shared__ float red[16][16];
  const int c = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int i = blockIdx.x * 16 + c;  // n is a multiple of 16
  float v = 0.f;
#pragma unroll 8
  for (int k = part; k < chunks; k += 16) v += partial[(int64_t)k * n + i];
  red[part][c] = v;
  __syncthreads();
  if (part) return;
#pragma unroll
  for (int p = 1; p < 16; ++p) v += red[p][c];
  out[i] = v;
}

// Rows of a chunk: 16, four a wave, until there are 128 chunks, then more.
static int64_t rows_per_chunk(int64_t M) { return M <= 2048 ? 16 : (M + 127) / 128; }

size_t grad_pre_workspace_bytes(int64_t M, int64_t N) {
  const int64_t rows = rows_per_chunk(M);
  return (size_t)((M + rows - 1) / rows) * (size_t)N * 4;
}

hipError_t launch_grad_pre(GradPreArgs a, hipStream_t stream) {
  a.chunk_rows = (int)rows_per_chunk(a.M);
  a.chunks = (a.M + a.chunk_rows - 1) / a.chunk_rows;
  if (a.M > 0) {
    const unsigned across = (unsigned)((grad_columns(a) + kCols - 1) / kCols);
    const dim3 grid(across, (unsigned)a.chunks);
    const bool shorts = a.chunk_rows <= 4 * kWaves;
    if (a.gated && shorts)
      grad_pre_kernel<true, 4><<<grid, 256, 0, stream>>>(a);
    else if (a.gated)
      grad_pre_kernel<true, 1><<<grid, 256, 0, stream>>>(a);
    else if (shorts)
      grad_pre_kernel<false, 4><<<grid, 256, 0, stream>>>(a);
    else
      grad_pre_kernel<false, 1><<<grid, 256, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.dbias) return hipSuccess;
  sum_chunks_kernel<<<(unsigned)(a.N / 16), 256, 0, stream>>>(a.partial, a.chunks, a.N, a.dbias);
  return hipGetLastError();
}

}  // namespace mxfp4
