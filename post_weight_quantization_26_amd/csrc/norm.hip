// Layer norm (rms: root-mean-square norm, mean taken as 0) of every token, for
// serving straight to the 8-bit rows of the next layer, and its gradient.
//
//   r = 1 / sqrt(mean_k (x - mean)² + eps),  xh = (x - mean)·r,  y = xh·gamma + beta
//
//   d = dy·gamma;  dx = r·(d - mean_k d [not rms] - xh·mean_k(d·xh))
//   dgamma = Σ_t dy·xh,  dbeta = Σ_t dy
#include "row_block.h"
#include "w8.h"

namespace awq {
namespace {

// gamma and beta, in X's type or float32.
template <int DT, int W>
__device__ __forceinline__ void load_weight(const void* g, bool f32, int K, int c, int t,
                                            float (&x)[8]) {
  if (DT != 0 && !f32) load_piece<DT, W>(g, 0, K, c, t, x);
  else load_piece<0, W>(g, 0, K, c, t, x);
}

// Bound by HBM: a row stays in registers over its three passes (sum, squares
// of deviations, output), so X is read once; gamma and beta come from L2.
template <int DT, int W, int V>
__global__ __launch_bounds__(kRowThreads<W>) void norm_kernel(const Norm p) {
  __shared__ float red0[16], red1[16];
  __shared__ uint32_t red2[16];
  const int64_t row = row_of<W>(blockIdx.x);
  if (row >= p.T) return;   // W = 1: no barrier follows; otherwise row < T
  const int t = row_thread<W>(), K = int(p.K);
  const int64_t at = row * K;
  float x[V][8];
#pragma unroll
  for (int c = 0; c < V; ++c) load_piece<DT, W>(p.X, at, K, c, t, x[c]);
  float mean = 0.f;
  if (!p.rms) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += x[c][e];
    mean = row_sum<W>(s, red0) / float(K);
  }
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < V; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (row_col<W>(c, t) + e < K) {
        x[c][e] -= mean;
        q = __builtin_fmaf(x[c][e], x[c][e], q);
      }
  const float rstd = 1.f / __builtin_sqrtf(row_sum<W>(q, red1) / float(K) + p.eps);
#pragma unroll
  for (int c = 0; c < V; ++c) {
    float g[8], b[8];
    load_weight<DT, W>(p.gamma, p.gamma32, K, c, t, g);
    if (p.beta) load_weight<DT, W>(p.beta, p.gamma32, K, c, t, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xh = x[c][e] * rstd;
      x[c][e] = p.beta ? __builtin_fmaf(xh, g[e], b[e]) : xh * g[e];
    }
    if (p.Y) store_piece<DT, W>(p.Y, at, K, c, t, x[c]);
  }
  if (p.stats && t == 0) *reinterpret_cast<float2*>(p.stats + 2 * row) = make_float2(mean, rstd);
  if (p.codes) quantize_row<W, V>(x, row, K, t, red2, p.codes, p.steps);
}

// Gradient, first launch. A group of waves takes every groups-th row and keeps
// its columns' sums of dy·xh and dy in registers, so dY and X are read once and
// dX written once; the groups' sums go to `partial` (float32), which a second
// launch adds up in a fixed order. A row's values are loaded one row ahead.
// Bound by HBM for long batches (8192 rows of 8192: 80 us, 5.0 TB/s, both launches), by
// the chain of a row's loads, sums and barrier for short ones.
//
// Up to 8192 columns a lane holds 8 of them and a group has as many waves as that
// takes, up to 16 (W): 8 waves of 16 columns a lane ran 1111 rows of 5000 in 30 us,
// 10 waves of 8 in 17, both launches. Above 8192 columns a lane holds 32 (V = 4), which
// for float32 do not fit its registers: 2000 rows of 16384 take 122 us (bf16 44), of
// 12001 99 (40); 16 waves of 16 a lane took 123 and 178. WHOLE: K is a multiple of 8.
//
// Only a lane's last piece can lie past a row's end: the others hold 512 columns for
// V = 2, which begins at 513, and 1536 for each 2048 that K begins for V = 4, which begins
// at 8193. That they are whole is known here spares their shifts (20000 rows of 777: 37
// -> 30 us; 2000 of 12001: float32 135 -> 99, bf16 48 -> 40).
template <int DT, int W, int V, bool WHOLE>
__global__ __launch_bounds__(V == 4 ? 512 : kRowThreads<W>) void norm_back_kernel(const NormBack p) {
  __shared__ float2 red[2][16];
  const int t = row_thread<W>(), K = int(p.K);
  const int64_t group = row_of<W>(blockIdx.x);
  if (group >= p.groups) return;   // W = 1 only: no barrier follows
  const float inv_k = 1.f / float(K);
  float g[V][8], ag[V][8] = {}, ab[V][8] = {};
#pragma unroll
  for (int c = 0; c < V; ++c) load_weight<DT, W>(p.gamma, p.gamma32, K, c, t, g[c]);
  Piece<DT> rx[V], ry[V];
  float2 st = make_float2(0.f, 0.f);
  int64_t row = group;
  auto load = [&](int64_t r) {
    if (r >= p.T) return;
    st = *reinterpret_cast<const float2*>(p.stats + 2 * r);
#pragma unroll
    for (int c = 0; c < V - 1; ++c) {
      rx[c].template load<W, true>(p.X, r * K, K, c, t);
      ry[c].template load<W, true>(p.dY, r * K, K, c, t);
    }
    rx[V - 1].template load<W, WHOLE, true>(p.X, r * K, K, V - 1, t);
    ry[V - 1].template load<W, WHOLE>(p.dY, r * K, K, V - 1, t);
  };
  load(row);
  for (int par = 0; row < p.T; row += p.groups, par ^= 1) {
    float xh[V][8], d[V][8], s1 = 0.f, s2 = 0.f;
    const float mean = p.rms ? 0.f : st.x, rstd = st.y;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      float x[8], dy[8];
      if (c < V - 1) {
        rx[c].template get<W, true>(K, c, t, x);
        ry[c].template get<W, true>(K, c, t, dy);
      } else {
        rx[c].template get<W, WHOLE, true>(K, c, t, x);
        ry[c].template get<W, WHOLE>(K, c, t, dy);
      }
      // past K, where d is 0, xh is one of the row's values or 0: -mean·r may be an
      // infinity, and 0 times it NaN
      const float m = c + 1 < V || row_col<W>(c, t) < K ? mean : 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[c][e] = (x[e] - m) * rstd;
        ag[c][e] = __builtin_fmaf(dy[e], xh[c][e], ag[c][e]);
        ab[c][e] += dy[e];
        d[c][e] = dy[e] * g[c][e];   // 0 past K
        s1 += d[c][e];
        s2 = __builtin_fmaf(d[c][e], xh[c][e], s2);
      }
    }
    load(row + p.groups);
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if constexpr (W > 1) {
      // a wave is back at this buffer two rows on, past the other's barrier
      if ((threadIdx.x & 63) == 0) red[par][threadIdx.x >> 6] = make_float2(s1, s2);
      __syncthreads();
      const unsigned i = threadIdx.x & 15;
      const float2 part = i < blockDim.x / 64 ? red[par][i] : make_float2(0.f, 0.f);
      s1 = row16_sum(part.x);
      s2 = row16_sum(part.y);
    }
    const float c1 = p.rms ? 0.f : s1 * inv_k, c2 = s2 * inv_k;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[e] = rstd * __builtin_fmaf(-xh[c][e], c2, d[c][e] - c1);
      store_piece<DT, W>(p.dX, row * K, K, c, t, o);
    }
  }
#pragma unroll
  for (int c = 0; c < V; ++c) {
    store_piece<0, W>(p.partial, group * p.Kp, K, c, t, ag[c]);
    if (p.dbeta)
      store_piece<0, W>(p.partial, (p.groups + group) * p.Kp, K, c, t, ab[c]);
  }
}

// Second launch: 64 columns of one of the two sums a workgroup, 16 lanes of 4
// columns each, the groups dealt to the 64 rows of lanes.
template <int DT>
__global__ __launch_bounds__(1024) void norm_sums_kernel(const float* __restrict__ partial,
                                                         int64_t groups, int64_t Kp, int K,
                                                         void* __restrict__ dgamma,
                                                         void* __restrict__ dbeta) {
  __shared__ float4 sum[64][16];
  const int lane = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int col = blockIdx.x * 64 + lane * 4;
  const float* base = partial + blockIdx.y * groups * Kp;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < Kp)
#pragma unroll 4
    for (int64_t r = part; r < groups; r += 64) {
      const float4 v = *reinterpret_cast<const float4*>(base + r * Kp + col);
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
  sum[part][lane] = a;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  const int c = threadIdx.x;
  float s[4] = {};
#pragma unroll
  for (int i = 0; i < 64; ++i) s[i & 3] += reinterpret_cast<const float*>(sum[i])[c];
  if (blockIdx.x * 64 + c < K)
    store1<DT>(blockIdx.y ? dbeta : dgamma, blockIdx.x * 64 + c, (s[0] + s[1]) + (s[2] + s[3]));
}

template <int DT, int W, int V>
hipError_t launch_fwd(const Norm& p, hipStream_t st) {
  norm_kernel<DT, W, V><<<row_grid<W, V>(p.T), row_block<W, V>(p.K), 0, st>>>(p);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_fwd_t(const Norm& p, hipStream_t st) {
  if (p.K <= 512) return launch_fwd<DT, 1, 1>(p, st);
  if (p.K <= 1024) return launch_fwd<DT, 1, 2>(p, st);
  // Up to a row a CU latency counts, and more waves of 8 columns a lane save some (33
  // rows of 4096: 4.0 instead of 4.5 us); else 16 a lane (28672 rows of 8192: 182
  // instead of 233, with 32 a lane 201).
  if (p.T <= 256 && p.K <= 8192) return launch_fwd<DT, 16, 1>(p, st);
  if (p.K <= 16384) return launch_fwd<DT, 16, 2>(p, st);
  return hipErrorInvalidValue;
}

template <int DT, int W, int V>
hipError_t launch_back(const NormBack& p, hipStream_t st) {
  const unsigned grid = row_grid<W, V>(p.groups), threads = row_block<W, V>(p.K);
  if (p.K % 8 == 0)
    norm_back_kernel<DT, W, V, true><<<grid, threads, 0, st>>>(p);
  else
    norm_back_kernel<DT, W, V, false><<<grid, threads, 0, st>>>(p);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_back_t(const NormBack& p, hipStream_t st) {
  if (p.K <= 512) return launch_back<DT, 1, 1>(p, st);
  if (p.K <= 1024) return launch_back<DT, 1, 2>(p, st);
  if (p.K <= 8192) return launch_back<DT, 16, 1>(p, st);
  if (p.K <= 16384) return launch_back<DT, 16, 4>(p, st);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_norm(const Norm& p, int dtype, hipStream_t st) {
  if (dtype == 0) return launch_fwd_t<0>(p, st);
  if (dtype == 1) return launch_fwd_t<1>(p, st);
  return launch_fwd_t<2>(p, st);
}

hipError_t launch_norm_back(const NormBack& p, int dtype, hipStream_t st) {
  hipError_t e = dtype == 0   ? launch_back_t<0>(p, st)
                 : dtype == 1 ? launch_back_t<1>(p, st)
                              : launch_back_t<2>(p, st);
  if (e != hipSuccess) return e;
  const dim3 grid(unsigned((p.K + 63) / 64), p.dbeta ? 2 : 1);
  const int odt = p.gamma32 ? 0 : dtype;
  if (odt == 0)
    norm_sums_kernel<0><<<grid, 1024, 0, st>>>(p.partial, p.groups, p.Kp, int(p.K), p.dgamma,
                                               p.dbeta);
  else if (odt == 1)
    norm_sums_kernel<1><<<grid, 1024, 0, st>>>(p.partial, p.groups, p.Kp, int(p.K), p.dgamma,
                                               p.dbeta);
  else
    norm_sums_kernel<2><<<grid, 1024, 0, st>>>(p.partial, p.groups, p.Kp, int(p.K), p.dgamma,
                                               p.dbeta);
  return hipGetLastError();
}

}  // namespace awq
