// Shared by the kernels of the 8-bit products (w8_*.hip).
#pragma once

#include "gemm_types.h"
#include "w8.h"
#include "w8_phi.h"

namespace awq {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));

// Codes: lane l supplies row (A) or column (B) l % 16 and 16 codes of the
// 64-wide contraction, those of lane group l / 16; it receives column l % 16
// and rows 4·(l / 16) + v. The sums are exact: |code| <= 128 and K < 2^17.
__device__ __forceinline__ intx4 mfma_16x16x64(intx4 a, intx4 b, intx4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// act(g) and, for the gradient, its derivative. exp and the reciprocal are the
// hardware's (1 ulp; the argument's rounding adds |g|·2^-23, all far below the
// output's 2^-8 or 2^-11); below 2^-126 both give zero, so that silu ends at g = -87.3,
// where it is -1e-36.
constexpr int kSilu = 0, kGelu = 1;
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-g));
}
// Φ(g) from e = exp(-g²/2): a fit of Φ / e for g <= 0 (w8_phi.h). The whole is within
// (1.5·g² + 14) of 2^-24, relative to the tail too down to float32's smallest normal
// numbers, the 1.5·g² from the exponent's argument. The library's erfc has branches that
// the gated epilogues pay for: 18 us more for each round of 256 tiles.
__device__ __forceinline__ float normal_cdf(float g, float e) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(g), kPhiT, 1.f));
  float q = kPhi[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) q = __builtin_fmaf(t, q, kPhi[i]);
  const float tail = e * (t * q);
  return g < 0.f ? tail : 1.f - tail;
}
template <int ACT>
__device__ __forceinline__ float act_of(float g) {
  if constexpr (ACT == kSilu) return g * sigmoid(g);
  return g * normal_cdf(g, __expf(-0.5f * g * g));
}
template <int ACT>
__device__ __forceinline__ float act_slope(float g, float& a) {
  if constexpr (ACT == kSilu) {
    const float s = sigmoid(g);
    a = g * s;
    return s * __builtin_fmaf(g, 1.f - s, 1.f);
  }
  const float e = __expf(-0.5f * g * g), cdf = normal_cdf(g, e);
  a = g * cdf;
  return __builtin_fmaf(g * 0.39894228040143268f, e, cdf);
}

template <bool F16>
__device__ __forceinline__ uint16_t round16(float f) {
  if constexpr (F16) return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
template <bool F16>
__device__ __forceinline__ float widen16(uint16_t h) {
  return F16 ? f16_to_f32(h) : bf16_to_f32(h);
}

// Four consecutive 16-bit outputs from o; vec: whole and 8-byte aligned.
template <bool F16>
__device__ __forceinline__ void store4(uint16_t* p, bool vec, int64_t left, const float (&y)[4]) {
  uint16_t h[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) h[v] = round16<F16>(y[v]);
  if (vec) {
    *reinterpret_cast<uint2*>(p) =
        make_uint2(uint32_t(h[0]) | uint32_t(h[1]) << 16, uint32_t(h[2]) | uint32_t(h[3]) << 16);
    return;
  }
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (v < left) p[v] = h[v];
}

// A product from its exact sum: one rounding of the sum to float32 (2^-24),
// then two float32 products.
__device__ __forceinline__ float scaled(int sum, float xs, float w) {
  return (float(sum) * xs) * w;
}

// The channels' side of the outputs n .. n + 3 (of N): steps and bias.
template <bool GATED>
struct Channels {
  float w[4], u[4], bias[4];
};
template <bool F16, bool GATED>
__device__ __forceinline__ Channels<GATED> channels(const W8Product& p, int64_t n) {
  Channels<GATED> c;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int64_t i = n + v < p.N ? n + v : p.N - 1;
    c.w[v] = p.w.steps[i];
    c.u[v] = GATED ? p.u.steps[i] : 0.f;
    c.bias[v] = !GATED && p.bias ? widen16<F16>(p.bias[i]) : 0.f;
  }
  return c;
}

// A tile's outputs: pointers at its first one, so that offsets within 256 rows of
// N (below 2^23) fit 32 bits.
struct Outputs {
  uint16_t *Y, *G, *U;
};
__device__ __forceinline__ Outputs outputs_at(const W8Product& p, int64_t t, int64_t n) {
  const int64_t o = t * p.N + n;
  return {p.Y + o, p.G ? p.G + o : nullptr, p.G ? p.U + o : nullptr};
}

// Outputs o .. o + 3 from their sums (and the second layer's), `left` of them valid.
template <bool F16, bool GATED, int ACT>
__device__ __forceinline__ void finish4(const Outputs& out, const Channels<GATED>& c, float xs,
                                        bool bias, uint32_t o, bool vec, int64_t left, intx4 s,
                                        intx4 su) {
  float y[4], u[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    y[v] = scaled(s[v], xs, c.w[v]);
    if constexpr (GATED) u[v] = scaled(su[v], xs, c.u[v]);
    else if (bias) y[v] += c.bias[v];
  }
  if constexpr (GATED) {
    if (out.G) {
      store4<F16>(out.G + o, vec, left, y);
      store4<F16>(out.U + o, vec, left, u);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) y[v] = act_of<ACT>(y[v]) * u[v];
  }
  store4<F16>(out.Y + o, vec, left, y);
}

}  // namespace
}  // namespace awq
