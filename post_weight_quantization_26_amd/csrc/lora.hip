// Low-rank adapters beside a packed 4-bit layer, forward and backward.
//
// Token t of X [T, K] uses adapter a = ids[t] of L (A_a [r, K], B_a [N, r],
// factor c_a); an id outside [0, L) is a token without one.
//
//   forward   h_t = A_a·x_t;  y_t = Ŵ·x_t + c_a·B_a·h_t
//   backward  g_t = c_a·B_aᵀ·dy_t;  dx_t = Ŵᵀ·dy_t + A_aᵀ·g_t
//             dA_a = Σ_{t of a} g_t·x_tᵀ;  dB_a = Σ_{t of a} c_a·dy_t·h_tᵀ
//
// with Ŵ[n][k] = (q[k][n] - z[k/g][n])·scale[k/g][n] of the layout that
// quantize_pack writes. Everything is summed in float32 and rounded once.
#include "lora.h"

namespace awq {
namespace {

template <bool F16>
__device__ __forceinline__ uint16_t to16(float f) {
  if constexpr (F16) return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
  else return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

template <bool F16>
__device__ __forceinline__ float from16(uint16_t h) {
  if constexpr (F16) return f16_to_f32(h);
  else return bf16_to_f32(h);
}

// Ŵ[n][k], exact in float32.
__device__ __forceinline__ float weight_at(const LoraLayer& w, int64_t n, int64_t k) {
  const int64_t N8 = w.N / 8, j = n >> 3, g = k / w.group;
  const int sh = 4 * int(n & 7);
  const float q = float((uint32_t(w.qweight[k * N8 + j]) >> sh) & 15u);
  const float z = float((uint32_t(w.qzeros[g * N8 + j]) >> sh) & 15u);
  return (q - z) * f16_to_f32(w.scales[g * w.N + n]);
}

// P[t][j] = f·Σ_c V[t][c]·M_a[j][c], f = c_a if SCALED. M_a is A_a [r, C]
// (ROWS) or B_a [C, r]. One workgroup per token, one wave per j at a time.
template <bool F16, bool ROWS, bool SCALED>
__global__ __launch_bounds__(256) void lora_down_kernel(const uint16_t* __restrict__ V, int64_t C,
                                                        LoraSet s,
                                                        const uint16_t* __restrict__ M,
                                                        float* __restrict__ P) {
  const int64_t t = blockIdx.x;
  const int a = s.ids[t], lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool has = a >= 0 && a < s.L;
  for (int j = wave; j < s.r; j += 4) {
    float sum = 0.f;
    if (has)
      for (int64_t c = lane; c < C; c += 64) {
        const int64_t m = ROWS ? (int64_t(a) * s.r + j) * C + c : (int64_t(a) * C + c) * s.r + j;
        sum = __builtin_fmaf(from16<F16>(V[t * C + c]), from16<F16>(M[m]), sum);
      }
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    if (SCALED && has) sum *= s.scaling[a];
    if (lane == 0) P[t * s.r + j] = sum;
  }
}

// O[t][o] = Σ_c V[t][c]·Ŵ(o, c) + f·Σ_j P[t][j]·U_a(o, j): the forward pass
// (o = n, c = k, U = B, f = c_a) or the backward one (BWD: o = k, c = n,
// U = Aᵀ, f = 1). 64 x 64 outputs per workgroup, 16 contraction steps in LDS.
template <bool F16, bool BWD>
__global__ __launch_bounds__(256) void lora_product_kernel(const uint16_t* __restrict__ V,
                                                           int64_t T, LoraLayer w, LoraSet s,
                                                           const float* __restrict__ P,
                                                           uint16_t* __restrict__ O) {
  __shared__ float vs[16][65], ws[16][65];
  const int64_t C = BWD ? w.N : w.K, W = BWD ? w.K : w.N;
  const int64_t t0 = int64_t(blockIdx.y) * 64, o0 = int64_t(blockIdx.x) * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t c0 = 0; c0 < C; c0 += 16) {
    for (int e = threadIdx.x; e < 64 * 16; e += 256) {
      const int c = e & 15, i = e >> 4;
      vs[c][i] = t0 + i < T && c0 + c < C ? from16<F16>(V[(t0 + i) * C + c0 + c]) : 0.f;
    }
    for (int e = threadIdx.x; e < 64 * 16; e += 256) {
      const int i = e & 63, c = e >> 6;
      const int64_t o = o0 + i, cc = c0 + c;
      ws[c][i] = o < W && cc < C ? weight_at(w, BWD ? cc : o, BWD ? o : cc) : 0.f;
    }
    __syncthreads();
    for (int c = 0; c < 16; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_fmaf(vs[c][ty + 16 * i], ws[c][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + ty + 16 * i;
    if (t >= T) continue;
    const int a = s.ids[t];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t o = o0 + tx + 16 * j;
      if (o >= W) continue;
      float y = acc[i][j];
      if (a >= 0 && a < s.L) {
        float e = 0.f;
        for (int q = 0; q < s.r; ++q) {
          const uint16_t u = BWD ? s.A[(int64_t(a) * s.r + q) * w.K + o]
                                 : s.B[(int64_t(a) * w.N + o) * s.r + q];
          e = __builtin_fmaf(P[t * s.r + q], from16<F16>(u), e);
        }
        y += BWD ? e : s.scaling[a] * e;
      }
      O[t * W + o] = to16<F16>(y);
    }
  }
}

}  // namespace

template <bool F16>
hipError_t forward_few(const LoraForward& p, hipStream_t st) {
  float* H = p.H ? p.H : p.P;
  lora_down_kernel<F16, true, false>
      <<<unsigned(p.T), 256, 0, st>>>(p.X, p.w.K, p.s, p.s.A, H);
  const dim3 grid(unsigned((p.w.N + 63) / 64), unsigned((p.T + 63) / 64));
  lora_product_kernel<F16, false><<<grid, 256, 0, st>>>(p.X, p.T, p.w, p.s, H, p.Y);
  if (!p.codes) return hipGetLastError();
  return launch_act_pack8(p.X, F16 ? 2 : 1, p.T, p.w.K, p.codes, p.steps, st);
}

hipError_t launch_lora_forward(const LoraForward& p, hipStream_t st) {
  if (p.T <= 16) return p.f16 ? forward_few<true>(p, st) : forward_few<false>(p, st);
  LoraDown d{};
  d.V = p.X;
  d.M = p.s.A;
  d.scaling = p.s.scaling;
  d.ids = p.s.ids;
  d.T = p.T;
  d.C = d.ldv = d.ldm = p.w.K;
  d.L = p.s.L;
  d.r = p.s.r;
  d.f16 = p.f16;
  d.H = p.H;
  d.Q = p.Q;
  d.RW = p.RW;
  d.E = p.E;
  d.codes = p.codes;
  d.steps = p.steps;
  hipError_t e = launch_lora_down(d, st);
  if (e != hipSuccess) return e;
  e = launch_w4a16_dequant(p.w.qweight, p.w.qzeros, p.w.scales, p.w.N, p.w.K, p.w.group, p.f16,
                           p.Wd, st);
  if (e != hipSuccess) return e;
  const LoraUp u{p.Q, p.E, p.s.ids, p.s.B, p.s.L, p.s.r, p.RW};
  return launch_lora_gemm(p.X, p.w.K, p.Wd, p.w.K, p.T, p.w.N, p.w.K, u, p.f16, p.Y, st);
}

}  // namespace awq
