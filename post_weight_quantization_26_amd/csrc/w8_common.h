// Shared by the kernels of the 8-bit products (w8_*.hip).
#pragma once

#include "gemm_types.h"
#include "w8.h"

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
// output's 2^-9 or 2^-12).
constexpr int kSilu = 0, kGelu = 1;
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-g));
}
template <int ACT>
__device__ __forceinline__ float act_of(float g) {
  if constexpr (ACT == kSilu) return g * sigmoid(g);
  // Φ(g) = erfc(-g / √2) / 2 keeps its digits where 1 + erf would cancel
  return g * (0.5f * erfcf(g * -0.70710678118654752f));
}
template <int ACT>
__device__ __forceinline__ float act_slope(float g, float& a) {
  if constexpr (ACT == kSilu) {
    const float s = sigmoid(g);
    a = g * s;
    return s * __builtin_fmaf(g, 1.f - s, 1.f);
  }
  const float cdf = 0.5f * erfcf(g * -0.70710678118654752f);
  a = g * cdf;
  return __builtin_fmaf(g * 0.39894228040143268f, __expf(-0.5f * g * g), cdf);
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

// A product from its exact sum: one rounding of the sum to float32 (2^-24),
// then two float32 products.
__device__ __forceinline__ float scaled(int sum, float xs, float w) {
  return (float(sum) * xs) * w;
}

}  // namespace
}  // namespace awq
