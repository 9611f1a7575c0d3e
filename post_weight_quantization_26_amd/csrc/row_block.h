// One row of a matrix in the registers of W waves: the loads, stores and
// reductions shared by the row quantiser (rows8.hip) and the norms (norm.hip).
//
// W is 1 (a workgroup of 4 waves holds 4 rows) or 4, 8, 16 (a workgroup is one
// row). A lane holds V pieces of 8 values. VEC: K is a multiple of 8 and every
// row 16-byte aligned, so a piece is 8 consecutive values; otherwise the 8
// values of a piece lie W·64 apart, so that a wave still reads consecutive
// elements.
#pragma once

#include "act8.h"
#include "device_common.h"

namespace awq {
namespace {

template <int DT>
__device__ __forceinline__ float load1(const void* base, int64_t i) {
  if constexpr (DT == 0) return static_cast<const float*>(base)[i];
  if constexpr (DT == 1) return bf16_to_f32(static_cast<const uint16_t*>(base)[i]);
  return f16_to_f32(static_cast<const uint16_t*>(base)[i]);
}

template <int DT>
__device__ __forceinline__ void store1(void* base, int64_t i, float v) {
  if constexpr (DT == 0)
    static_cast<float*>(base)[i] = v;
  else if constexpr (DT == 1)
    static_cast<uint16_t*>(base)[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else
    static_cast<uint16_t*>(base)[i] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

template <int W>
constexpr int kRowThreads = W < 4 ? 256 : W * 64;

// Thread t of a row's W·64, its row among the workgroup's.
template <int W>
__device__ __forceinline__ int row_thread() {
  return W == 1 ? int(threadIdx.x & 63) : int(threadIdx.x);
}
template <int W>
__device__ __forceinline__ int64_t row_of(int64_t block) {
  return W == 1 ? block * 4 + (threadIdx.x >> 6) : block;
}

template <int W, bool VEC>
__device__ __forceinline__ int row_col(int c, int e, int t) {
  return VEC ? (c * (W * 64) + t) * 8 + e : (c * 8 + e) * (W * 64) + t;
}

// Columns past K are zero.
template <int DT, int W, bool VEC>
__device__ __forceinline__ void load_piece(const void* base, int64_t at, int K, int c, int t,
                                           float (&x)[8]) {
  if constexpr (VEC) {
    if (row_col<W, VEC>(c, 0, t) < K) {
      load8<DT>(base, at + row_col<W, VEC>(c, 0, t), x);
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int col = row_col<W, VEC>(c, e, t);
      x[e] = col < K ? load1<DT>(base, at + col) : 0.f;
    }
  }
}

template <int DT, int W, bool VEC>
__device__ __forceinline__ void store_piece(void* base, int64_t at, int K, int c, int t,
                                            const float (&x)[8]) {
  if constexpr (VEC) {
    if (row_col<W, VEC>(c, 0, t) < K) store8<DT>(base, at + row_col<W, VEC>(c, 0, t), x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int col = row_col<W, VEC>(c, e, t);
      if (col < K) store1<DT>(base, at + col, x[e]);
    }
  }
}

template <int W, bool VEC>
__device__ __forceinline__ void store_codes(int8_t* base, int64_t at, int K, int c, int t,
                                            uint2 codes) {
  if constexpr (VEC) {
    if (row_col<W, VEC>(c, 0, t) < K)
      *reinterpret_cast<uint2*>(base + at + row_col<W, VEC>(c, 0, t)) = codes;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int col = row_col<W, VEC>(c, e, t);
      if (col < K) base[at + col] = int8_t((e < 4 ? codes.x : codes.y) >> (8 * (e & 3)));
    }
  }
}

// v summed over a wave, the same bits in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#define AWQ_ROR_ADD(N)                                                                         \
  v += __uint_as_float(uint32_t(                                                               \
      __builtin_amdgcn_update_dpp(0, int(__float_as_uint(v)), 0x120 + N, 0xF, 0xF, false)));
  AWQ_ROR_ADD(8) AWQ_ROR_ADD(4) AWQ_ROR_ADD(2) AWQ_ROR_ADD(1)
#undef AWQ_ROR_ADD
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    s[i] = __uint_as_float(
        uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(v)), 16 * i)));
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
  m = row16_max(m);
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = uint32_t(__builtin_amdgcn_readlane(int(m), 16 * i));
    r = r > u ? r : u;
  }
  return r;
}

// Over a row's W waves. `red` holds W values and is used for one reduction of
// the workgroup only (or again after another barrier in between).
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (W == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) s += red[i];
  return s;
}
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* red) {
  m = wave_max(m);
  if constexpr (W == 1) return m;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) r = r > red[i] ? r : red[i];
  return r;
}

// The row's codes and step from its values.
template <int W, int V, bool VEC>
__device__ __forceinline__ void quantize_row(const float (&x)[V][8], int64_t row, int K, int t,
                                             uint32_t* red, int8_t* codes, float* steps) {
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const uint32_t u = act8_abs_max(x[c]);
    m = m > u ? m : u;
  }
  const Act8Scale s = act8_scale(row_max<W>(m, red));
  const int64_t at = row * K;
#pragma unroll
  for (int c = 0; c < V; ++c)
    store_codes<W, VEC>(codes, at, K, c, t, act8_codes(x[c], s));
  if (t == 0) steps[row] = s.step;
}

}  // namespace
}  // namespace awq
