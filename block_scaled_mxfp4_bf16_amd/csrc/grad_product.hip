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

// 128 x 128 outputs a workgroup, 64 x 64 a wave, 32 of j a stage.
template <bool TRANSPOSED>
__global__ __launch_bounds__(256) void grad_product_kernel(const GradProductArgs a) {
  constexpr int BI = 128, BK = 128, BJ = 32;
  __shared__ __attribute__((aligned(16))) uint8_t p_lds[BI * BJ * 2];
  __shared__ __attribute__((aligned(16))) uint8_t t_lds[BK * BJ * 2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i0 = blockIdx.x * BI, k0 = blockIdx.y * BK;
  const int wi = (wave & 1) * 64, wk = (wave >> 1) * 64;
  const int gp = ((a.K >> 5) + 7) & ~7;
  const int stages = (a.J + BJ - 1) / BJ;
  const int first = blockIdx.z * a.split_stages;
  const int last = first + a.split_stages < stages ? first + a.split_stages : stages;

  v16f acc[2][2];  // [32 of k][32 of i]
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.f;

  for (int s = first; s < last; ++s) {
    const int j0 = s * BJ;
    __syncthreads();
    // P: 512 chunks of 16 bytes
#pragma unroll
    for (int c = tid; c < BI * BJ / 8; c += 256) {
      u32x4 v = {0, 0, 0, 0};
      if (TRANSPOSED) {
        const int j = c / (BI / 8), q = c % (BI / 8);
        if (j0 + j < a.J && i0 + 8 * q < a.I) v = *(const u32x4 *)(a.P + (int64_t)(j0 + j) * a.ldp + i0 + 8 * q);
        *(u32x4 *)(p_lds + turned_at(j, q, BI * 2)) = v;
      } else {
        const int i = c / (BJ / 8), q = c % (BJ / 8);
        if (i0 + i < a.I && j0 + 8 * q < a.J) v = *(const u32x4 *)(a.P + (int64_t)(i0 + i) * a.ldp + j0 + 8 * q);
        *(u32x4 *)(p_lds + i * (BJ * 2) + ((q ^ ((i >> 1) & 3)) << 4)) = v;
      }
    }
    // T: 128 chunks of a row's 32 codes
    if (tid < BJ * BK / 32) {
      const int r = tid & 15, t = (tid >> 4) % (BK / 32), gg = (tid >> 4) / (BK / 32);
      const int g = (j0 >> 4) + gg, grp = (k0 >> 5) + t;
      u32x4 w = {0, 0, 0, 0};
      float scale = 0.f;
      if (16 * g < a.J && grp < (a.K >> 5)) {
        w = *(const u32x4 *)(a.codes + ((int64_t)g * (a.K >> 5) + grp) * 256 + r * 16);
        const uint32_t byte =
            a.scales[(int64_t)(g >> 1) * 32 * gp + shuffled_scale_offset((g & 1) * 16 + r, grp, gp)];
        scale = __uint_as_float(byte << 23);
      }
      const int j = gg * 16 + r;
#pragma unroll
      for (int q = 0; q < 4; ++q) *(u32x4 *)(t_lds + turned_at(j, 4 * t + q, BK * 2)) = bf16_of_codes(w[q], scale);
    }
    __syncthreads();
#pragma unroll
    for (int ss = 0; ss < 2; ++ss) {
      const int jr = ss * 16 + (lane >> 5) * 8 + ((lane & 15) >> 2);  // the lane's row of turned reads
      const auto turned = [&](const uint8_t *m, int col, int row_bytes) {
        // columns col + lane % 32, rows 8 * (lane / 32) .. + 7 of the half stage
        const int c = (col + ((lane >> 4) & 1) * 16 + (lane & 3) * 4) * 2;
        const int at = (c & 15);
        return join(read_turned(m + turned_at(jr, c >> 4, row_bytes) + at),
                    read_turned(m + turned_at(jr + 4, c >> 4, row_bytes) + at));
      };
      bf16x8 tf[2], pf[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        tf[x] = turned(t_lds, wk + 32 * x, BK * 2);
        if (TRANSPOSED) {
          pf[x] = turned(p_lds, wi + 32 * x, BI * 2);
        } else {
          const int i = wi + 32 * x + (lane & 31), q = ss * 2 + (lane >> 5);
          pf[x] = *(const bf16x8 *)(p_lds + i * (BJ * 2) + ((q ^ ((i >> 1) & 3)) << 4));
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(tf[x], pf[y], acc[x][y], 0, 0, 0);
    }
  }
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int i = i0 + wi + 32 * y + (lane & 31);
    if (i >= a.I) continue;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int k = k0 + wk + 32 * x + 8 * p + 4 * (lane >> 5);
        if (k >= a.K) continue;
        const v4f v = {acc[x][y][4 * p], acc[x][y][4 * p + 1], acc[x][y][4 * p + 2], acc[x][y][4 * p + 3]};
        if (a.splits > 1)
          *(v4f *)(a.partial + ((int64_t)blockIdx.z * a.I + i) * a.K + k) = v;
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
  const int64_t tiles = ((I + 127) / 128) * ((K + 127) / 128), most = J / 256;
  const int64_t want = 256 / tiles;
  const int64_t s = want < most ? want : most;
  return s < 1 ? 1 : s;
}

size_t grad_product_workspace_bytes(int64_t I, int64_t J, int64_t K) {
  const int64_t s = splits_of(I, J, K);
  return s > 1 ? (size_t)s * (size_t)I * (size_t)K * 4 : 0;
}

hipError_t launch_grad_product(GradProductArgs a, hipStream_t stream) {
  const int stages = (a.J + 31) / 32;
  const int64_t want = splits_of(a.I, a.J, a.K);
  a.split_stages = (int)((stages + want - 1) / want);
  a.splits = a.split_stages > 0 ? (stages + a.split_stages - 1) / a.split_stages : 1;
  const dim3 grid((a.I + 127) / 128, (a.K + 127) / 128, a.splits);
  if (a.transposed)
    grad_product_kernel<true><<<grid, 256, 0, stream>>>(a);
  else
    grad_product_kernel<false><<<grid, 256, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits <= 1) return e;
  const int64_t quads = (int64_t)a.I * (a.K / 4);
  join_splits_kernel<<<(unsigned)((quads + 255) / 256), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace mxfp4
