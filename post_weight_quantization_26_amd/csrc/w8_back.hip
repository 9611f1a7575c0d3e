// Gradient of the 8-bit products with respect to their input (taken as the
// values that its 8-bit rows stand for):
//
//   plain   dx[t][k] = Σ_n (dy[t][n]·w_n)·q[n][k]
//   gated   dg = dh·u·act'(g), du = dh·act(g);
//           dx[t][k] = Σ_n (dg·wg_n)·qg[n][k] + Σ_n (du·wu_n)·qu[n][k]
//
// One 16-bit product: the steps join the gradient in the operand A [T, C] (one
// rounding), the codes are exact operands B [K, C] in either type. A pair's
// two sums are one contraction of twice the length. Three launches: A, B, and
// the 256x256 main loop of gemm_core.h.
#include "gemm_core.h"
#include "w8_common.h"

namespace awq {
namespace {

// A row of A. fp16: dy·w may leave the type's range, so the row is divided by
// the power of two that takes its largest finite value below 2^14, which the
// last launch multiplies back in (exactly, but for results below 2^-126); a
// first pass finds it. Columns from N to Np are zero.
template <bool F16, bool GATED, int ACT>
__global__ __launch_bounds__(256) void w8_grad_rows_kernel(const W8Back p) {
  __shared__ uint32_t red[4];
  const int64_t t = blockIdx.x;
  const uint16_t* dy = p.dY + t * p.N;
  const uint16_t* gr = GATED ? p.G + t * p.N : nullptr;
  const uint16_t* ur = GATED ? p.U + t * p.N : nullptr;
  uint16_t* out = p.A + t * (GATED ? 2 : 1) * p.Np;
  auto values = [&](int64_t n, float& a, float& b, float& dg, float& du) {
    const float d = widen16<F16>(dy[n]);
    if constexpr (GATED) {
      const float u = widen16<F16>(ur[n]);
      float ac;
      const float slope = act_slope<ACT>(widen16<F16>(gr[n]), ac);
      dg = (d * u) * slope;
      du = d * ac;
      a = dg * p.w.steps[n];
      b = du * p.u.steps[n];
    } else {
      a = d * p.w.steps[n];
      b = 0.f;
    }
  };
  float scale = 1.f;
  if constexpr (F16) {
    uint32_t m = 0;
    for (int64_t n = threadIdx.x; n < p.N; n += 256) {
      float a, b, dg, du;
      values(n, a, b, dg, du);
      const uint32_t ua = __float_as_uint(a) & 0x7FFFFFFFu, ub = __float_as_uint(b) & 0x7FFFFFFFu;
      if (ua < 0x7F800000u && ua > m) m = ua;
      if (ub < 0x7F800000u && ub > m) m = ub;
    }
#pragma unroll
    for (int i = 32; i; i >>= 1) {
      const uint32_t o = __shfl_xor(m, i);
      m = m > o ? m : o;
    }
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) m = m > red[i] ? m : red[i];
    // 2^e <= largest < 2^(e+1): divide by 2^(e-13); the factor and its inverse
    // stay normal numbers
    int e = int(m >> 23) - 127 - 13;
    e = e < -126 ? -126 : e > 126 ? 126 : e;
    scale = m ? __uint_as_float(uint32_t(127 - e) << 23) : 1.f;
    if (threadIdx.x == 0) p.E[t] = m ? __uint_as_float(uint32_t(127 + e) << 23) : 1.f;
  }
  for (int64_t n = threadIdx.x; n < p.Np; n += 256) {
    float a = 0.f, b = 0.f, dg, du;
    if (n < p.N) {
      values(n, a, b, dg, du);
      if constexpr (GATED) {
        p.dG[t * p.N + n] = round16<F16>(dg);
        p.dU[t * p.N + n] = round16<F16>(du);
      }
    }
    out[n] = round16<F16>(a * scale);
    if constexpr (GATED) out[p.Np + n] = round16<F16>(b * scale);
  }
}

// B: 64 x 64 codes through LDS, as 16-bit numbers. grid (Np / 64, K / 64, layers).
template <bool F16>
__global__ __launch_bounds__(256) void w8_transpose_kernel(const W8Back p, int64_t C) {
  __shared__ uint32_t tile[64][17];   // [n][k / 4]
  const int64_t n0 = int64_t(blockIdx.x) * 64, k0 = int64_t(blockIdx.y) * 64;
  const int8_t* q = blockIdx.z ? p.u.q : p.w.q;
  const int r = threadIdx.x >> 2, c = threadIdx.x & 3;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (n0 + r < p.N) v = *reinterpret_cast<const uint4*>(q + (n0 + r) * p.K + k0 + c * 16);
  tile[r][c * 4] = v.x;
  tile[r][c * 4 + 1] = v.y;
  tile[r][c * 4 + 2] = v.z;
  tile[r][c * 4 + 3] = v.w;
  __syncthreads();
  // row k of B: 16 consecutive n a thread
  const int k = threadIdx.x >> 2, nn = (threadIdx.x & 3) * 16;
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int8_t lo = int8_t(tile[nn + 2 * i][k >> 2] >> (8 * (k & 3)));
    const int8_t hi = int8_t(tile[nn + 2 * i + 1][k >> 2] >> (8 * (k & 3)));
    h[i] = uint32_t(round16<F16>(float(lo))) | uint32_t(round16<F16>(float(hi))) << 16;
  }
  uint4* o = reinterpret_cast<uint4*>(p.B + (k0 + k) * C + int64_t(blockIdx.z) * p.Np + n0 + nn);
  o[0] = make_uint4(h[0], h[1], h[2], h[3]);
  o[1] = make_uint4(h[4], h[5], h[6], h[7]);
}

// dX = E·(A·Bᵀ): the main loop's A rows are the channels k, so a lane holds 4
// consecutive ones of a token.
template <bool F16>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(1, 1)))
void w8_back_gemm_kernel(const W8Back p, int64_t C, int tiles_t, int tiles_k) {
  int tt, tk;
  if (!tile_of(blockIdx.x, tiles_t, tiles_k, tt, tk)) return;
  const int64_t t0 = int64_t(tt) * BN, k0 = int64_t(tk) * BM;
  const int64_t rows_k = p.K - k0 < BM ? p.K - k0 : BM;
  const int64_t rows_t = p.T - t0 < BN ? p.T - t0 : BN;
  GemmCtx64 c;
  gemm_setup64(c, p.B + k0 * C, rows_k, p.A + t0 * C, rows_t, C);
  floatx4 acc[8][8];
  gemm_mainloop16<F16>(c, acc);
  const int lane = threadIdx.x & 63;
  const int wm = c.wave >> 1, wn = c.wave & 1;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t t = t0 + wn * 128 + j * 16 + (lane & 15);
    if (t >= p.T) continue;
    const float e = F16 ? p.E[t] : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t k = k0 + wm * 128 + i * 16 + 4 * (lane >> 4);
      if (k >= p.K) continue;   // K is a multiple of 128
      uint16_t h[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) h[v] = round16<F16>(acc[i][j][v] * e);
      *reinterpret_cast<uint2*>(p.dX + t * p.K + k) =
          make_uint2(uint32_t(h[0]) | uint32_t(h[1]) << 16, uint32_t(h[2]) | uint32_t(h[3]) << 16);
    }
  }
}

template <bool F16>
hipError_t launch_back(const W8Back& p, hipStream_t st) {
  const bool gated = p.G != nullptr;
  const int64_t C = (gated ? 2 : 1) * p.Np;
  const unsigned rows = unsigned(p.T);
  if (!gated) w8_grad_rows_kernel<F16, false, kSilu><<<rows, 256, 0, st>>>(p);
  else if (p.act == kSilu) w8_grad_rows_kernel<F16, true, kSilu><<<rows, 256, 0, st>>>(p);
  else w8_grad_rows_kernel<F16, true, kGelu><<<rows, 256, 0, st>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid(unsigned(p.Np / 64), unsigned(p.K / 64), gated ? 2 : 1);
  w8_transpose_kernel<F16><<<grid, 256, 0, st>>>(p, C);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int tiles_t = int((p.T + BN - 1) / BN), tiles_k = int((p.K + BM - 1) / BM);
  w8_back_gemm_kernel<F16><<<unsigned(gemm_blocks(tiles_t, tiles_k)), NT, 0, st>>>(p, C, tiles_t,
                                                                                 tiles_k);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w8_back(const W8Back& p, hipStream_t st) {
  return p.f16 ? launch_back<true>(p, st) : launch_back<false>(p, st);
}

}  // namespace awq
