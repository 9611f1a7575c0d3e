// Activation checkpoints in 8 bits: one step per token and 128 channels.
//
//   m = max(max |x|, 2^-100);  step = fl32(m / 127);  inv = fl32(127 / m)
//   code = rint(fl32(x·inv));  x^ = fl32(code·step)
//
// |x|·inv exceeds 127 by at most one rounding, so |code| <= 127 without a
// clamp; 2^-100 keeps inv finite. A block that holds a NaN or an infinity
// gets the step NaN and codes 0, so all of it comes back as NaN.
#include "lora.h"

namespace awq {
namespace {

template <int DT>
__device__ __forceinline__ float load1(const void* X, int64_t i) {
  if constexpr (DT == 0) return static_cast<const float*>(X)[i];
  else if constexpr (DT == 1) return bf16_to_f32(static_cast<const uint16_t*>(X)[i]);
  else return f16_to_f32(static_cast<const uint16_t*>(X)[i]);
}

template <int DT>
__device__ __forceinline__ void store1(void* X, int64_t i, float f) {
  if constexpr (DT == 0) static_cast<float*>(X)[i] = f;
  else if constexpr (DT == 1)
    static_cast<uint16_t*>(X)[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
  else static_cast<uint16_t*>(X)[i] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
}

// One wave per block of 128 channels, two channels per lane.
template <int DT>
__global__ __launch_bounds__(256) void act_pack8_kernel(const void* __restrict__ X, int64_t blocks,
                                                        int8_t* __restrict__ codes,
                                                        float* __restrict__ steps) {
  const int64_t b = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (b >= blocks) return;
  float x[2];
  uint32_t m = 0;   // |x| as bits: infinities and NaN compare above every finite value
  for (int i = 0; i < 2; ++i) {
    x[i] = load1<DT>(X, b * 128 + lane + 64 * i);
    const uint32_t u = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    m = m > u ? m : u;
  }
  for (int o = 32; o; o >>= 1) {
    const uint32_t u = __shfl_xor(m, o);
    m = m > u ? m : u;
  }
  const bool finite = m < 0x7F800000u;
  const float mx = fmaxf(__uint_as_float(m), 0x1p-100f);
  const float inv = 127.f / mx;
  for (int i = 0; i < 2; ++i)
    codes[b * 128 + lane + 64 * i] =
        finite ? int8_t(int(__builtin_rintf(x[i] * inv))) : int8_t(0);
  if (lane == 0) steps[b] = finite ? mx / 127.f : __uint_as_float(0x7FC00000u);
}

template <int DT>
__global__ __launch_bounds__(256) void act_unpack8_kernel(const int8_t* __restrict__ codes,
                                                          const float* __restrict__ steps,
                                                          int64_t n, void* __restrict__ X) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) store1<DT>(X, i, float(codes[i]) * steps[i / 128]);
}

}  // namespace

hipError_t launch_act_pack8(const void* X, int dtype, int64_t T, int64_t K, int8_t* codes,
                            float* steps, hipStream_t st) {
  const int64_t blocks = T * (K / 128);
  const unsigned grid = unsigned((blocks + 3) / 4);
  if (dtype == 0) act_pack8_kernel<0><<<grid, 256, 0, st>>>(X, blocks, codes, steps);
  else if (dtype == 1) act_pack8_kernel<1><<<grid, 256, 0, st>>>(X, blocks, codes, steps);
  else act_pack8_kernel<2><<<grid, 256, 0, st>>>(X, blocks, codes, steps);
  return hipGetLastError();
}

hipError_t launch_act_unpack8(const int8_t* codes, const float* steps, int dtype, int64_t T,
                              int64_t K, void* X, hipStream_t st) {
  const int64_t n = T * K;
  const unsigned grid = unsigned((n + 255) / 256);
  if (dtype == 0) act_unpack8_kernel<0><<<grid, 256, 0, st>>>(codes, steps, n, X);
  else if (dtype == 1) act_unpack8_kernel<1><<<grid, 256, 0, st>>>(codes, steps, n, X);
  else act_unpack8_kernel<2><<<grid, 256, 0, st>>>(codes, steps, n, X);
  return hipGetLastError();
}

}  // namespace awq
