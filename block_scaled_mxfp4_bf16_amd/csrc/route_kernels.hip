// The router of a mixture-of-experts block:
//   g[t, e]   softmax over e, or sigmoid, of the logits
//   ids[t]    the k experts of the largest g + bias, in falling order, ties to
//             the lower expert; an expert whose logit or bias is -inf or NaN
//             is never chosen (id -1, weight 0 once none is left)
//   w[t, j]   g of the chosen, divided by their sum if asked
// and the stable sort of the (token, choice) pairs by expert: offsets[e], the
// pair at each sorted place (rows) and the place of each pair (pos).
//
// The choice is made on whole numbers: a value maps to an unsigned integer of
// the same order, so the largest is a plain integer maximum.  Without a bias
// the logits themselves order the experts (both scores rise with the logit);
// with one, an f32 estimate of g + bias orders them, and wherever two are
// closer than its error the f64 values decide, since two f32 sums that round
// to the same value would pick the wrong expert.  L lanes share a token, L = 16
// wherever E <= 256 and k <= 16: a maximum over 16 lanes is four rotate steps
// and serves four tokens of a wave at once.  The weights of the k chosen are
// computed in f64, one lane each, and rounded once.
//
// The k maxima depend on each other, and that chain bounds it, not memory: 8192
// tokens of 128 experts, sigmoid with a bias, k 8, take 11.6 us to choose (4 MB of
// logits; least 10.9) and 6.8 to place; one token of 64 experts 5.2 us, one launch.
#include <type_traits>

#include "experts_bounds.hpp"
#include "experts_device.hpp"
#include "experts_internal.hpp"

namespace mxfp4 {

namespace {

// The value of lane (l + N) % 16 of the lane's row of 16.
template <int N>
__device__ __forceinline__ uint32_t rotate16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 | N, 0xF, 0xF, false);
}

// All-reduce over groups of L lanes; `op` on u32, u64 or double values.
template <int N, class T>
__device__ __forceinline__ T rotated(T v) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, rotate16<N>(__builtin_bit_cast(uint32_t, v)));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint64_t r = rotate16<N>((uint32_t)u) | ((uint64_t)rotate16<N>((uint32_t)(u >> 32)) << 32);
    return __builtin_bit_cast(T, r);
  }
}
template <int L, class T, class Op>
__device__ __forceinline__ T all_reduce(T v, Op op) {
  v = op(v, rotated<8>(v));
  v = op(v, rotated<4>(v));
  v = op(v, rotated<2>(v));
  v = op(v, rotated<1>(v));
  if constexpr (L >= 32) v = op(v, (T)__shfl_xor(v, 16));
  if constexpr (L >= 64) v = op(v, (T)__shfl_xor(v, 32));
  return v;
}

// Integers in the order of the values; 0 stands for "never chosen" and is
// below every finite value's.  -0 counts as 0.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ uint64_t order_of(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  return b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}

// A logit as f32; +inf counts as the largest finite value, NaN as -inf.
__device__ __forceinline__ float logit(const RouteArgs &a, int64_t row, int e) {
  const int64_t at = row * a.ld + e;
  float v;
  if (a.x_type == MXFP4_TYPE_F32)
    v = ((const float *)a.logits)[at];
  else if (a.x_type == MXFP4_TYPE_BF16)
    v = (float)((const __bf16 *)a.logits)[at];
  else
    v = (float)((const _Float16 *)a.logits)[at];
  return v != v ? -__builtin_inff() : __builtin_fminf(v, 3.402823466e38f);
}

__device__ __forceinline__ bool lowest(float v) { return v == -__builtin_inff(); }

// Value of an integer of order_of(float), never 0.
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// One token by the L lanes of the caller's group (V experts a lane, expert
// l + L * v).  Lane j < k returns choice j.
template <int L, int V, bool BIAS>
__device__ __forceinline__ void route_token(const RouteArgs &a, int64_t t, int l, int *id_out, float *w_out) {
  const auto larger = [](auto p, auto q) { return p > q ? p : q; };
  const auto smaller = [](int p, int q) { return p < q ? p : q; };
  const auto plus = [](auto p, auto q) { return p + q; };
  const bool softmax = a.score == MXFP4_SCORE_SOFTMAX;
  float x[V], bias[BIAS ? V : 1];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = l + L * v;
    x[v] = e < a.E ? logit(a, t, e) : -__builtin_inff();
    if constexpr (BIAS) bias[v] = e < a.E ? a.bias[e] : 0.f;
  }
  float top = 0.f;  // of the softmax
  if (softmax) {
    top = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) top = larger(top, x[v]);
    top = all_reduce<L>(top, larger);
    if (lowest(top)) top = 0.f;
  }
  const auto sum64 = [&]() {
    double s = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) s += exp((double)x[v] - top);
    return all_reduce<L>(s, plus);
  };
  // renormalized weights need no sum over all experts
  const double total = softmax && !a.renorm ? sum64() : 1.0;

  // Without a bias the key is the logit's own.  With one it is that of an f32
  // estimate of g + bias.  Two of them are out of order only where they are
  // closer than 2^-18 + 2^-22 of the larger, which is what decides below whether
  // f64 is asked: the addition is off by 2^-24 of its result, and g by less than
  // 2^-19 = 32 u, u = 2^-24 (hardware exponential and reciprocal: 1 ulp, 2 u).
  //   sigmoid  e = exp(-x) is off by (1.5 |x| + 2) u e; g (1 - g) of that, at most
  //            0.9 u, 1 + e rounds once and the reciprocal: 4 u together.
  //   softmax  g = exp(d) / s, d = x - top <= 0.  Its own exponential: (2.5 |d| +
  //            2) u g with |d| exp(d) < 0.37, the reciprocal 2 u, the product 1 u,
  //            the sum's V - 1 + log2(L) <= 21 additions 21 u g.  The exponentials
  //            summed add (2 + 2.5 a) u g, a = sum of g |d|, which is at most
  //            h(g) + (1 - g) ln 1024 (h the entropy of g and 1 - g): largest all
  //            together near g = 1, where a is next to 0: below 29 u.
  uint32_t key[V];
  if constexpr (BIAS) {
    float g[V];
#pragma unroll
    for (int v = 0; v < V; ++v) g[v] = softmax ? __expf(x[v] - top) : __builtin_amdgcn_rcpf(1.0f + __expf(-x[v]));
    float scale = 1.f;
    if (softmax) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) s += g[v];
      s = all_reduce<L>(s, plus);
      scale = s > 0.f ? __builtin_amdgcn_rcpf(s) : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool dead = lowest(x[v]) || lowest(bias[v]) || bias[v] != bias[v];
      key[v] = dead ? 0 : order_of(__builtin_fminf(g[v] * scale + bias[v], 3.402823466e38f));
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = lowest(x[v]) ? 0 : order_of(x[v]);
  }

  int id = -1;
  double sum_all = 0.0;  // of the softmax, once two estimates are too close
  for (int j = 0; j < a.k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = larger(m, key[v]);
    m = all_reduce<L>(m, larger);
    int c = INT32_MAX;
    if constexpr (BIAS) {
      const float top_value = value_of(m ? m : 0x80000000u);
      const uint32_t below = order_of(top_value - (0x1p-18f + 0x1p-22f * __builtin_fabsf(top_value)));
      const uint32_t near = m && below ? below : 1u;  // keys from here on may be the largest
      int n = 0;
#pragma unroll
      for (int v = V - 1; v >= 0; --v) {
        const bool is = key[v] >= near;
        n += is;
        c = is ? l + L * v : c;
      }
      const uint64_t with = __ballot(n != 0) >> (__lane_id() & (64 - L));
      const int lanes = __builtin_popcountll(L == 64 ? with : with & ((1ull << (L & 63)) - 1));
      c = all_reduce<L>(c, smaller);
      if (__ballot(n > 1 || lanes > 1)) {
        // more than one candidate in some token of the wave: decide by f64
        if (softmax && sum_all == 0.0) sum_all = sum64();
        uint64_t best = 0;
        int at = INT32_MAX;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (__ballot(key[v] >= near)) {
            const double g = softmax ? exp((double)x[v] - top) / sum_all : 1.0 / (1.0 + exp(-(double)x[v]));
            const uint64_t o = key[v] >= near ? order_of(g + bias[v]) : 0;
            at = o > best ? l + L * v : at;
            best = larger(best, o);
          }
        }
        const uint64_t all = all_reduce<L>(best, larger);
        const int exact = all_reduce<L>(best == all ? at : INT32_MAX, smaller);
        c = m ? exact : c;
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = l + L * v == c ? 0 : key[v];
      } else {
        // the one candidate of each token
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = key[v] >= near ? 0 : key[v];
      }
    } else {
#pragma unroll
      for (int v = V - 1; v >= 0; --v) c = key[v] == m ? l + L * v : c;
      c = all_reduce<L>(c, smaller);
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = l + L * v == c ? 0 : key[v];
    }
    if (l == j) id = m ? c : -1;
  }

  double w = 0.0;
  if (id >= 0) {
    const double xl = (double)logit(a, t, id);
    w = softmax ? exp(xl - top) / total : 1.0 / (1.0 + exp(-xl));
  }
  if (a.renorm) {
    const double s = all_reduce<L>(w, plus);
    w = s > 0.0 ? w / s : w;
  }
  *id_out = id;
  *w_out = (float)w;
}

// Tokens [t0, t1) by the block's groups of L lanes: ids and weights, and the
// count of each expert in `hist` (zeroed by the caller).
template <int L, int V, bool BIAS, int THREADS>
__device__ __forceinline__ void route_tokens(const RouteArgs &a, int64_t t0, int64_t t1, int *hist) {
  const int l = threadIdx.x & (L - 1);
  for (int64_t t = t0 + threadIdx.x / L; t < t1; t += THREADS / L) {
    int id;
    float w;
    route_token<L, V, BIAS>(a, t, l, &id, &w);
    if (l < a.k) {
      a.ids[t * a.k + l] = id;
      a.weights[t * a.k + l] = w;
      if (id >= 0) atomicAdd(&hist[id], 1);
    }
  }
}

// Exclusive sums of v[0 .. E), in place, by one wave.
__device__ __forceinline__ int scan_experts(int *v, int E) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) >> 6;
  const int lo = lane * per < E ? lane * per : E;
  const int hi = lo + per < E ? lo + per : E;
  int s = 0;
  for (int e = lo; e < hi; ++e) s += v[e];
  int incl = s;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  int run = incl - s;
  for (int e = lo; e < hi; ++e) {
    const int c = v[e];
    v[e] = run;
    run += c;
  }
  return __shfl(incl, 63);
}

// Sorted places of the pairs [p0, p1): each wave of the block takes a
// contiguous run of them, counts its experts, and then walks its run 64 pairs
// at a time; lanes of the same expert find each other by ballots over the
// bits of the id.  next[e] is the first free place of expert e.
template <int THREADS>
__device__ __forceinline__ void place_pairs(const RouteArgs &a, int64_t p0, int64_t p1, const int *next,
                                            int (*wave_next)[kRouteMaxExperts]) {
  const int pairs = a.T * a.k;
  constexpr int W = THREADS / 64;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int64_t run = ((p1 - p0 + W - 1) / W + 63) / 64 * 64;
  const int64_t lo = p0 + wave * run, hi = lo + run < p1 ? lo + run : p1;
  for (int i = threadIdx.x; i < W * a.E; i += THREADS) wave_next[i / a.E][i % a.E] = 0;
  __syncthreads();
  for (int64_t p = lo + lane; p < hi; p += 64) {
    const int id = a.ids[p];
    if (id >= 0) atomicAdd(&wave_next[wave][id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += THREADS) {
    int at = next[e];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int c = wave_next[w][e];
      wave_next[w][e] = at;
      at += c;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(a.E);  // of every id below E
  for (int64_t p = lo; p < hi; p += 64) {
    const int64_t mine = p + lane;
    const int id = mine < hi ? a.ids[mine] : -1;
    uint64_t same = __ballot(id >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((id >> b) & 1);
      same &= (id >> b) & 1 ? set : ~set;
    }
    const int before = __builtin_popcountll(same & ((1ull << lane) - 1));
    if (id >= 0) {
      const int at = wave_next[wave][id] + before;
      // always, unless another call has written to the counts
      if ((unsigned)at < (unsigned)pairs) a.rows[at] = (int32_t)mine;
      a.pos[mine] = at;
    } else if (mine < hi) {
      a.pos[mine] = -1;
    }
    wave_lds_fence();
    if (id >= 0 && before == 0) wave_next[wave][id] += __builtin_popcountll(same);
    wave_lds_fence();
  }
}

}  // namespace

// First launch of many tokens: block b takes tokens [b * per_block, ...) and
// leaves its count of expert e in hist[e][b] (16 bits: a token takes an expert
// once, and a block has at most 4096 tokens).
template <int L, int V, bool BIAS>
__global__ __launch_bounds__(512) void route_choose_kernel(const RouteArgs a) {
  __shared__ int hist[kRouteMaxExperts];
  for (int e = threadIdx.x; e < a.E; e += 512) hist[e] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * a.per_block;
  route_tokens<L, V, BIAS, 512>(a, t0, t0 + a.per_block < a.T ? t0 + a.per_block : a.T, hist);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += 512) a.hist[((int64_t)e << a.hist_shift) + blockIdx.x] = (uint16_t)hist[e];
}

// Second launch: the same blocks add up the counts before theirs and place
// their pairs.  Every block reads all counts, 16 bytes (8 blocks of one
// expert) a load, 8 loads in flight: one a lane and dependent, as in a plain
// loop, they took 30 us of the 35 of 256 blocks of 128 experts.
__global__ __launch_bounds__(512) void route_place_kernel(const RouteArgs a) {
  __shared__ int next[kRouteMaxExperts];    // all counts, then first place, of each expert
  __shared__ int before[kRouteMaxExperts];  // pairs of the expert in earlier blocks
  __shared__ int wave_next[8][kRouteMaxExperts];
  __shared__ int used;
  for (int e = threadIdx.x; e < a.E; e += 512) next[e] = before[e] = 0;
  __syncthreads();
  // 16 lanes share an expert where it has 16 chunks of 8 blocks or more
  const int per_expert = a.hist_shift - 3;  // log2 of its chunks
  const int chunks = a.E << per_expert;
  for (int c0 = 0; c0 < chunks; c0 += 512 * 8) {
    u32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + 512 * i + threadIdx.x;
      v[i] = c < chunks ? ((const u32x4 *)a.hist)[c] : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + 512 * i + threadIdx.x;
      const int e = c >> per_expert;
      const int b0 = (c - (e << per_expert)) * 8;
      int all = 0, mine = 0;
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const int n = (v[i][h >> 1] >> (16 * (h & 1))) & 0xFFFF;
        all += b0 + h < a.blocks ? n : 0;
        mine += b0 + h < (int)blockIdx.x ? n : 0;
      }
      if (per_expert >= 4) {
        all = all_reduce<16>(all, [](int p, int q) { return p + q; });
        mine = all_reduce<16>(mine, [](int p, int q) { return p + q; });
        if ((threadIdx.x & 15) != 0) continue;
      }
      if (c < chunks) {
        atomicAdd(&next[e], all);
        atomicAdd(&before[e], mine);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int n = scan_experts(next, a.E);
    if (threadIdx.x == 0) used = within(n, 0, a.T * a.k);
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < a.E; e += 512) a.offsets[e] = next[e];
    if (threadIdx.x == 0) a.offsets[a.E] = used;
  }
  const int64_t pairs = (int64_t)a.T * a.k;
  for (int64_t p = used + (int64_t)blockIdx.x * 512 + threadIdx.x; p < pairs; p += (int64_t)a.blocks * 512)
    a.rows[p] = -1;
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += 512) next[e] += before[e];
  const int64_t p0 = (int64_t)blockIdx.x * a.per_block * a.k;
  const int64_t p1 = p0 + (int64_t)a.per_block * a.k;
  place_pairs<512>(a, p0, p1 < pairs ? p1 : pairs, next, wave_next);
}

// Few tokens: all of it in one workgroup and one launch.
template <int L, int V, bool BIAS>
__global__ __launch_bounds__(512) void route_small_kernel(const RouteArgs a) {
  __shared__ int next[kRouteMaxExperts];
  __shared__ int wave_next[8][kRouteMaxExperts];
  __shared__ int used;
  for (int e = threadIdx.x; e < a.E; e += 512) next[e] = 0;
  __syncthreads();
  route_tokens<L, V, BIAS, 512>(a, 0, a.T, next);
  __syncthreads();  // the ids this block wrote are read back below
  if (threadIdx.x < 64) {
    const int n = scan_experts(next, a.E);
    if (threadIdx.x == 0) used = within(n, 0, a.T * a.k);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += 512) a.offsets[e] = next[e];
  if (threadIdx.x == 0) a.offsets[a.E] = used;
  const int pairs = a.T * a.k;
  for (int p = used + threadIdx.x; p < pairs; p += 512) a.rows[p] = -1;
  place_pairs<512>(a, 0, pairs, next, wave_next);
}

// Up to this many tokens one workgroup does everything.
constexpr int kSmallTokens = 128;

// Tokens per block otherwise: at most 256 blocks, whole passes of 16 tokens.
static int64_t route_per_block(int64_t T) { return ((T + 255) / 256 + 15) / 16 * 16; }

// log2 of the places per expert in the counts: a power of two that holds all
// blocks, 8 at least.
static int route_hist_shift(int64_t T) {
  const int64_t per = route_per_block(T), blocks = (T + per - 1) / per;
  int s = 3;
  while ((1 << s) < blocks) ++s;
  return s;
}

size_t route_workspace_bytes(int64_t T, int64_t E) {
  return T <= kSmallTokens ? 0 : (size_t)(E << route_hist_shift(T)) * 2;
}

template <int L, int V, bool BIAS>
static hipError_t run_route(RouteArgs a, hipStream_t stream) {
  if (a.T <= kSmallTokens) {
    route_small_kernel<L, V, BIAS><<<1, 512, 0, stream>>>(a);
    return hipGetLastError();
  }
  a.per_block = (int)route_per_block(a.T);
  a.blocks = (a.T + a.per_block - 1) / a.per_block;
  a.hist_shift = route_hist_shift(a.T);
  route_choose_kernel<L, V, BIAS><<<a.blocks, 512, 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  route_place_kernel<<<a.blocks, 512, 0, stream>>>(a);
  return hipGetLastError();
}

template <bool BIAS>
static hipError_t run_route_layout(const RouteArgs &a, hipStream_t stream) {
  if (a.k <= 16) {
    if (a.E <= 64) return run_route<16, 4, BIAS>(a, stream);
    if (a.E <= 128) return run_route<16, 8, BIAS>(a, stream);
    if (a.E <= 256) return run_route<16, 16, BIAS>(a, stream);
  } else if (a.E <= 256) {
    return run_route<32, 8, BIAS>(a, stream);
  }
  return run_route<64, 16, BIAS>(a, stream);
}

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
  return a.bias ? run_route_layout<true>(a, stream) : run_route_layout<false>(a, stream);
}

}  // namespace mxfp4
