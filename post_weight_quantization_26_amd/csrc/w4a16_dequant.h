// The dequantisation of a packed 4-bit layer into [N, K] operand rows (w4a16.hip;
// beside other work, lora_down.hip): Ŵ = (q - z)·scale in float32, rounded once.
#pragma once

#include "device_common.h"

namespace awq {
namespace {

template <bool F16>
__device__ __forceinline__ uint16_t to16(float f) {
  if constexpr (F16) return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
  else return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

// The 8 fp16 scales of output channels 8j..8j+7 in group g (16 bytes) and
// their 8 zero points (one packed word) as float32.
__device__ __forceinline__ void group_params(const int32_t* __restrict__ qzeros,
                                             const uint16_t* __restrict__ scales, int64_t N,
                                             int64_t g, int64_t j, float (&sc)[8],
                                             float (&zf)[8]) {
  const uint4 s4 = *reinterpret_cast<const uint4*>(scales + g * N + 8 * j);
  const uint32_t sw[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sc[2 * i] = f16_to_f32(uint16_t(sw[i] & 0xFFFFu));
    sc[2 * i + 1] = f16_to_f32(uint16_t(sw[i] >> 16));
  }
  const uint32_t zw = uint32_t(qzeros[g * (N / 8) + j]);
#pragma unroll
  for (int r = 0; r < 8; ++r) zf[r] = float((zw >> (4 * r)) & 0xFu);
}

// Lane (kb, j): k rows 8kb..8kb+7 of word column j -> 8 output rows x 8 k,
// one 16-byte store per output row (consecutive lanes continue the same row).
template <bool F16>
__device__ __forceinline__ void dequant_words(int64_t t, const int32_t* __restrict__ qweight,
                                   const int32_t* __restrict__ qzeros,
                                   const uint16_t* __restrict__ scales, int64_t N, int64_t K,
                                   int group, uint16_t* __restrict__ Wd) {
#pragma clang fp contract(off)
  const int64_t K8 = K / 8, N8 = N / 8;
  if (t >= K8 * N8) return;
  const int64_t kb = t % K8, j = t / K8;
  const int64_t k0 = kb * 8;
  float sc[8], zf[8];
  group_params(qzeros, scales, N, k0 / group, j, sc, zf);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = uint32_t(qweight[(k0 + i) * N8 + j]);
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = (float((w[2 * i] >> (4 * r)) & 0xFu) - zf[r]) * sc[r];
      const float hi = (float((w[2 * i + 1] >> (4 * r)) & 0xFu) - zf[r]) * sc[r];
      h[i] = uint32_t(to16<F16>(lo)) | (uint32_t(to16<F16>(hi)) << 16);
    }
    *reinterpret_cast<uint4*>(Wd + (8 * j + r) * K + k0) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// N a multiple of 32: lane (kb, j) takes k rows 8kb..8kb+7 of word columns
// 4j..4j+3 (output rows 32j..32j+31) with one 16-byte load per k row, so a
// 128-byte line of qweight feeds 8 lanes instead of 32.
template <bool F16>
__device__ __forceinline__ void dequant_words4(int64_t t, const int32_t* __restrict__ qweight,
                                   const int32_t* __restrict__ qzeros,
                                   const uint16_t* __restrict__ scales, int64_t N, int64_t K,
                                   int group, uint16_t* __restrict__ Wd) {
#pragma clang fp contract(off)
  const int64_t K8 = K / 8, N8 = N / 8, N32 = N / 32;
  if (t >= K8 * N32) return;
  const int64_t kb = t % K8, j = t / K8;
  const int64_t k0 = kb * 8, g = k0 / group;
  uint4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint4*>(qweight + (k0 + i) * N8 + 4 * j);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float sc[8], zf[8];
    group_params(qzeros, scales, N, g, 4 * j + c, sc, zf);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = c == 0 ? w[2 * i].x : c == 1 ? w[2 * i].y : c == 2 ? w[2 * i].z : w[2 * i].w;
        const uint32_t b = c == 0 ? w[2 * i + 1].x : c == 1 ? w[2 * i + 1].y
                         : c == 2 ? w[2 * i + 1].z : w[2 * i + 1].w;
        const float lo = (float((a >> (4 * r)) & 0xFu) - zf[r]) * sc[r];
        const float hi = (float((b >> (4 * r)) & 0xFu) - zf[r]) * sc[r];
        h[i] = uint32_t(to16<F16>(lo)) | (uint32_t(to16<F16>(hi)) << 16);
      }
      *reinterpret_cast<uint4*>(Wd + (32 * j + 8 * c + r) * K + k0) =
          make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}

}  // namespace
}  // namespace awq
