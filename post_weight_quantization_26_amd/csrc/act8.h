// The arithmetic of an 8-bit activation checkpoint (act8.hip), shared with the
// kernel that makes one on its way through X (lora_down.hip).
#pragma once

#include "device_common.h"

namespace awq {

struct Act8 {
  uint2 codes;   // the lane's 8 codes, lowest byte first
  float step;    // the block's step
};

// A block's step and reciprocal from the bits of its largest |x| (as bits,
// infinities and NaN compare above every finite value).
struct Act8Scale {
  float step, inv;
  bool finite;
};
__device__ __forceinline__ Act8Scale act8_scale(uint32_t max_bits) {
#pragma clang fp contract(off)
  Act8Scale s;
  s.finite = max_bits < 0x7F800000u;
  const float m = fmaxf(__uint_as_float(max_bits), 0x1p-100f);
  s.inv = 127.f / m;
  s.step = s.finite ? m / 127.f : __uint_as_float(0x7FC00000u);
  return s;
}

__device__ __forceinline__ uint32_t act8_abs_max(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t u = __float_as_uint(x[e]) & 0x7FFFFFFFu;
    m = m > u ? m : u;
  }
  return m;
}

__device__ __forceinline__ uint2 act8_codes(const float (&x)[8], const Act8Scale& s) {
#pragma clang fp contract(off)
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int q = s.finite ? int(__builtin_rintf(x[e] * s.inv)) : 0;
    w[e >> 2] |= (uint32_t(q) & 0xFFu) << (8 * (e & 3));
  }
  return make_uint2(w[0], w[1]);
}

// max of m over the 16 lanes of a DPP row, in every lane
__device__ __forceinline__ uint32_t row16_max(uint32_t m) {
  uint32_t u;
#define AWQ_ROR_MAX(N)                                                              \
  u = uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x120 + N, 0xF, 0xF, false)); \
  m = m > u ? m : u;
  AWQ_ROR_MAX(8) AWQ_ROR_MAX(4) AWQ_ROR_MAX(2) AWQ_ROR_MAX(1)
#undef AWQ_ROR_MAX
  return m;
}

// 8 channels of a block whose largest |x| `reduce` finds over its lanes.
template <class Reduce>
__device__ __forceinline__ Act8 act8_block(const float (&x)[8], const Reduce& reduce) {
  const Act8Scale s = act8_scale(reduce(act8_abs_max(x)));
  return {act8_codes(x, s), s.step};
}

}  // namespace awq
