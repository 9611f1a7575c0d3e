// Activation checkpoints in 8 bits: one step per token and 128 channels.
//
//   m = max(max |x|, 2^-100);  step = fl32(m / 127);  inv = fl32(127 / m)
//   code = rint(fl32(x·inv));  x^ = fl32(code·step)
//
// |x|·inv exceeds 127 by at most one rounding, so |code| <= 127 without a
// clamp; 2^-100 keeps inv finite. A block that holds a NaN or an infinity
// gets the step NaN and codes 0, so all of it comes back as NaN.
#include "act8.h"
#include "lora.h"

namespace awq {
namespace {

// Bound by HBM: pack reads X once and writes 1.03 bytes an element, unpack
// the reverse. A lane takes 8 consecutive channels (one 16-byte load of a
// 16-bit type, one 8-byte store of codes), 16 lanes a block of 128, so the
// block's maximum is four DPP steps within a row of 16 lanes. A thread takes
// kActUnroll such pieces a workgroup apart, all loaded before any is used.
// fp16 32768x8192: pack 151 to 162 us (5.0 to 5.4 TB/s), unpack 124 (6.6, part of it
// from the cache behind L2); 129x4096: 3.6 and 2.8 us.
constexpr int kActUnroll = 4;

template <int DT>
__device__ __forceinline__ void store8(void* X, int64_t i, const float (&v)[8]) {
  if constexpr (DT == 0) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(X) + i);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (DT == 1)
        w[e] = uint32_t(__builtin_bit_cast(uint16_t, static_cast<__bf16>(v[2 * e]))) |
               uint32_t(__builtin_bit_cast(uint16_t, static_cast<__bf16>(v[2 * e + 1]))) << 16;
      else
        w[e] = uint32_t(__builtin_bit_cast(uint16_t, static_cast<_Float16>(v[2 * e]))) |
               uint32_t(__builtin_bit_cast(uint16_t, static_cast<_Float16>(v[2 * e + 1]))) << 16;
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(X) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// n8 = pieces of 8 channels; a block is 16 pieces, so whole rows of 16 lanes
// are in or out of range together.
template <int DT>
__global__ __launch_bounds__(256) void act_pack8_kernel(const void* __restrict__ X, int64_t n8,
                                                        int8_t* __restrict__ codes,
                                                        float* __restrict__ steps) {
  const int64_t p0 = int64_t(blockIdx.x) * (256 * kActUnroll) + threadIdx.x;
  float x[kActUnroll][8];
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u)
    if (p0 + 256 * u < n8) load8<DT>(X, (p0 + 256 * u) * 8, x[u]);
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    const int64_t p = p0 + 256 * u;
    if (p >= n8) break;
    const Act8 q = act8_block(x[u], [](uint32_t m) { return row16_max(m); });
    *reinterpret_cast<uint2*>(codes + p * 8) = q.codes;
    if ((p & 15) == 0) steps[p >> 4] = q.step;
  }
}

template <int DT>
__global__ __launch_bounds__(256) void act_unpack8_kernel(const int8_t* __restrict__ codes,
                                                          const float* __restrict__ steps,
                                                          int64_t n8, void* __restrict__ X) {
  const int64_t p0 = int64_t(blockIdx.x) * (256 * kActUnroll) + threadIdx.x;
  uint2 c[kActUnroll];
  float s[kActUnroll];
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u)
    if (p0 + 256 * u < n8) {
      c[u] = *reinterpret_cast<const uint2*>(codes + (p0 + 256 * u) * 8);
      s[u] = steps[(p0 + 256 * u) >> 4];
    }
#pragma unroll
  for (int u = 0; u < kActUnroll; ++u) {
    if (p0 + 256 * u >= n8) break;
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = float(int8_t(c[u].x >> (8 * e))) * s[u];
      v[4 + e] = float(int8_t(c[u].y >> (8 * e))) * s[u];
    }
    store8<DT>(X, (p0 + 256 * u) * 8, v);
  }
}

}  // namespace

// At most 2^34 elements: 2^31 pieces, 2^29 threads.
hipError_t launch_act_pack8(const void* X, int dtype, int64_t T, int64_t K, int8_t* codes,
                            float* steps, hipStream_t st) {
  const int64_t n8 = T * K / 8;
  const unsigned grid = unsigned((n8 + 256 * kActUnroll - 1) / (256 * kActUnroll));
  if (dtype == 0) act_pack8_kernel<0><<<grid, 256, 0, st>>>(X, n8, codes, steps);
  else if (dtype == 1) act_pack8_kernel<1><<<grid, 256, 0, st>>>(X, n8, codes, steps);
  else act_pack8_kernel<2><<<grid, 256, 0, st>>>(X, n8, codes, steps);
  return hipGetLastError();
}

hipError_t launch_act_unpack8(const int8_t* codes, const float* steps, int dtype, int64_t T,
                              int64_t K, void* X, hipStream_t st) {
  const int64_t n8 = T * K / 8;
  const unsigned grid = unsigned((n8 + 256 * kActUnroll - 1) / (256 * kActUnroll));
  if (dtype == 0) act_unpack8_kernel<0><<<grid, 256, 0, st>>>(codes, steps, n8, X);
  else if (dtype == 1) act_unpack8_kernel<1><<<grid, 256, 0, st>>>(codes, steps, n8, X);
  else act_unpack8_kernel<2><<<grid, 256, 0, st>>>(codes, steps, n8, X);
  return hipGetLastError();
}

}  // namespace awq
