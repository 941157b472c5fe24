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
// chunk.  The bias' gradient is summed in f32 by each lane over its rows, over
// the waves in LDS, and over the chunks by a second launch, in that order.
__global__ __launch_bounds__(256) void grad_pre_kernel(const GradPreArgs a) {
  __shared__ __attribute__((aligned(16))) v4f red[2][kWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = a.N >> 1;
  const int cols = a.gated ? half : a.N;
  const int col = blockIdx.x * kCols + lane * 4;
  const bool live = col < cols;
  const int first = blockIdx.y * a.chunk_rows;
  const int last = first + a.chunk_rows < a.M ? first + a.chunk_rows : a.M;
  v4f sum = {0.f, 0.f, 0.f, 0.f}, sum_up = {0.f, 0.f, 0.f, 0.f};
  if (live)
    for (int row = first + wave; row < last; row += kWaves) {
      const v4f dy = load4(a.dy, a.dy_type, (int64_t)row * a.ld_dy + col, a.wide);
      v4f dz = dy;
      if (a.pre) {
        const v4f z = load4(a.pre, 0, (int64_t)row * a.ld_pre + col, a.wide);
        v4f f, slope;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float s;
          f[i] = activate_slope(a.act, z[i], s);
          slope[i] = s;
        }
        dz = dy * slope;
        if (a.gated) {
          dz = dz * load4(a.pre, 0, (int64_t)row * a.ld_pre + half + col, a.wide);
          const v4f dup = dy * f;
          store4(a.dz, 0, (int64_t)row * a.ld_dz + half + col, dup, a.wide);
          sum_up += dup;
        }
      }
      store4(a.dz, 0, (int64_t)row * a.ld_dz + col, dz, a.wide);
      sum += dz;
    }
  if (!a.dbias) return;
  red[0][wave][lane] = sum;
  red[1][wave][lane] = sum_up;
  __syncthreads();
  if (wave < (a.gated ? 2 : 1) && live) {
    v4f v = red[wave][0][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += red[wave][w][lane];
    *(v4f *)(a.partial + (int64_t)blockIdx.y * a.N + wave * half + col) = v;
  }
}

__global__ __launch_bounds__(256) void sum_chunks_kernel(const float *partial, int chunks, int n, float *out) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.f;
  for (int c = 0; c < chunks; ++c) v += partial[(int64_t)c * n + i];
  out[i] = v;
}

// Rows of a chunk: enough chunks to fill the chip, no more than 128 of them.
static int64_t rows_per_chunk(int64_t M) { return M <= 512 ? 16 : (M + 127) / 128 < 16 ? 16 : (M + 127) / 128; }

size_t grad_pre_workspace_bytes(int64_t M, int64_t N) {
  const int64_t rows = rows_per_chunk(M);
  return (size_t)((M + rows - 1) / rows) * (size_t)N * 4;
}

hipError_t launch_grad_pre(GradPreArgs a, hipStream_t stream) {
  a.chunk_rows = (int)rows_per_chunk(a.M);
  a.chunks = (a.M + a.chunk_rows - 1) / a.chunk_rows;
  if (a.M > 0) {
    const unsigned across = (unsigned)((grad_columns(a) + kCols - 1) / kCols);
    grad_pre_kernel<<<dim3(across, (unsigned)a.chunks), 256, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.dbias) return hipSuccess;
  sum_chunks_kernel<<<(unsigned)((a.N + 255) / 256), 256, 0, stream>>>(a.partial, a.chunks, a.N, a.dbias);
  return hipGetLastError();
}

}  // namespace mxfp4
