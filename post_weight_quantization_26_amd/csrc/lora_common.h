// Device helpers of the low-rank adapter kernels.
#pragma once

#include "device_common.h"

namespace awq {
namespace {

template <bool F16>
__device__ __forceinline__ uint16_t round16(float f) {
  if constexpr (F16) return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
  else return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

template <bool F16>
__device__ __forceinline__ float widen16(uint16_t h) {
  if constexpr (F16) return f16_to_f32(h);
  else return bf16_to_f32(h);
}

// Two float32 values rounded to nearest even into a packed 16-bit pair, low
// half first, by a vector conversion, which is one instruction (two casts
// are four). Not inline asm: the compiler would put no wait states between
// that and an MFMA that reads the result.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
  typedef _Float16 h16x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  if constexpr (F16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, h16x2));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b16x2));
}

// The exponent e of a float32 magnitude in [2^e, 2^(e+1)), clamped to what leaves
// 2^(14-e), 2^-e and 2^e normal numbers (0: the least, what is not finite: the largest).
constexpr int kLeastExponent = -112, kLargestExponent = 126;
__device__ __forceinline__ int exponent_of(float m) {
  const int e = int((__float_as_uint(m) >> 23) & 0xFFu) - 127;
  return e < kLeastExponent ? kLeastExponent : e > kLargestExponent ? kLargestExponent : e;
}

__device__ __forceinline__ float exp2i(int e) {   // 2^e, -126 <= e <= 127
  return __uint_as_float(uint32_t(e + 127) << 23);
}

}  // namespace
}  // namespace awq
