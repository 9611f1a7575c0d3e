// Matrix-core operand types and the compiler's 16x16x32 MFMA, for kernels
// that leave hazards and register classes to the compiler.
#pragma once

#include <hip/hip_runtime.h>

namespace awq {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

// MFMA operand vector of 8 elements: bf16 or fp16 (F16 = true).
template <bool F16>
struct Operand {
  typedef bf16x8_t type;
};
template <>
struct Operand<true> {
  typedef f16x8_t type;
};

// Lane l supplies row (A) or column (B) l % 16, elements 8·(l / 16) .. + 7 of
// the 32-wide contraction; it receives column l % 16 and rows 4·(l / 16) + v.
__device__ __forceinline__ floatx4 mfma_16x16x32(bf16x8_t a, bf16x8_t b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mfma_16x16x32(f16x8_t a, f16x8_t b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

}  // namespace
}  // namespace awq
