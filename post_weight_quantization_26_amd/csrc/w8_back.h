// Shared by the two forms of the 8-bit products' gradient (w8_back.hip,
// w8_back_few.hip).
#pragma once

#include "row_block.h"
#include "w8_common.h"

namespace awq {

// dX from A in operand order (w8_back_few.hip).
hipError_t launch_w8_back_few(const W8Back& p, hipStream_t st);

namespace {

typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));

// Two codes as exact fp16 numbers. sel picks one byte of `lo` into the low half
// and the same byte of `hi` into the high half, the upper bytes zero (0x0C):
// v_perm_b32 numbers lo's bytes 0 .. 3 and hi's 4 .. 7. A byte's sign bit flipped
// is the code + 128, and under the exponent of 1024 (0x6400) the number
// 1024 + 128 + code; taking 1152 off is exact.
__device__ __forceinline__ uint32_t codes_to_f16(uint32_t lo, uint32_t hi, uint32_t sel) {
  const uint32_t u = __builtin_amdgcn_perm(hi, lo, sel) ^ 0x64806480u;
  const halfx2 v = __builtin_bit_cast(halfx2, u) - halfx2{_Float16(1152), _Float16(1152)};
  return __builtin_bit_cast(uint32_t, v);
}
// byte b of both
constexpr uint32_t byte_pair(int b) { return 0x0C040C00u + 0x00010001u * uint32_t(b); }

}  // namespace
}  // namespace awq
