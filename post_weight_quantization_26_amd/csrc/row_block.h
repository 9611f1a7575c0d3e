// One row of a matrix in the registers of W waves: the loads, stores and
// reductions shared by the row quantiser (rows8.hip) and the norms (norm.hip).
//
// W is 1 (a workgroup of 4 waves holds 4 rows, a wave each) or 16 (a workgroup is one
// row, of as many waves as it takes, up to 16). A lane holds V pieces of 8 consecutive
// values, which one or two loads of 16 bytes bring wherever the row starts: global
// memory takes them at any element's address, and rows of odd lengths run nearly as
// fast as aligned ones. Only a row's last piece, if it is not whole, is stored element
// by element.
#pragma once

#include "act8.h"
#include "device_common.h"

namespace awq {
namespace {

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
constexpr int kRowThreads = W == 1 ? 256 : 1024;   // at most
// Workgroups of T rows of K, and their threads.
template <int W, int V>
inline unsigned row_grid(int64_t T) {
  return unsigned(W == 1 ? (T + 3) / 4 : T);
}
template <int W, int V>
inline unsigned row_block(int64_t K) {
  return W == 1 ? 256 : unsigned((K + 512 * V - 1) / (512 * V)) * 64;
}

// A thread's number among its row's, its row among the workgroup's.
template <int W>
__device__ __forceinline__ int row_thread() {
  return W == 1 ? int(threadIdx.x & 63) : int(threadIdx.x);
}
template <int W>
__device__ __forceinline__ int64_t row_of(int64_t block) {
  return W == 1 ? block * 4 + (threadIdx.x >> 6) : block;
}

// First column of a thread's piece c.
template <int W>
__device__ __forceinline__ int row_col(int c, int t) {
  return (c * (W == 1 ? 64 : int(blockDim.x)) + t) * 8;
}

// 16 or 8 bytes at any address.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
template <int DT>
__device__ __forceinline__ const char* element(const void* base, int64_t i) {
  return static_cast<const char*>(base) + i * (DT == 0 ? 4 : 2);
}

// A piece as loaded, columns past K zero (SAME: within a row's last piece, not whole, some
// of its values again). A row's last piece, if it is not whole, loads
// the row's last 8 elements and moves them down when they are read: element by element
// the load itself would wait for its parts (1111 rows of 5003, gradient: 34 -> 31 us).
template <int DT>
struct Piece {
  static constexpr int kWords = DT == 0 ? 8 : 4, kEach = 8 / kWords;   // elements a word
  uint32_t w[kWords];

  // WHOLE: the piece is within the row or past it as a whole
  template <int W, bool WHOLE = false, bool SAME = false>
  __device__ __forceinline__ void load(const void* base, int64_t at, int K, int c, int t) {
    const int col = row_col<W>(c, t);
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
    if (!WHOLE && K < 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (SAME ? col >= K : col + e >= K) continue;
        const int64_t i = at + (SAME && col + e >= K ? K - 1 : col + e);
        if constexpr (DT == 0) w[e] = static_cast<const uint32_t*>(base)[i];
        else w[e >> 1] |= uint32_t(static_cast<const uint16_t*>(base)[i]) << (16 * (e & 1));
      }
    } else if (col < K) {
      const char* p = element<DT>(base, at + (col + 8 <= K ? col : K - 8));
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = load16(p + 4 * i);
        w[i] = v.x;
        w[i + 1] = v.y;
        w[i + 2] = v.z;
        w[i + 3] = v.w;
      }
    }
  }

  template <int W, bool WHOLE = false, bool SAME = false>
  __device__ __forceinline__ void get(int K, int c, int t, float (&x)[8]) const {
    uint32_t u[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) u[i] = w[i];
    if (!WHOLE && (K & 7) && K > 8) {   // else every piece is whole, or loaded in place
      const int past = row_col<W>(c, t) + 8 - K, n = past > 0 && past < 8 ? past : 0;
      if constexpr (kEach == 2) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          const uint32_t next = i + 1 < kWords ? u[i + 1] : SAME ? u[i] : 0;
          u[i] = n & 1 ? __builtin_amdgcn_alignbit(next, u[i], 16) : u[i];
        }
      }
#pragma unroll
      for (int step = 1; step < kWords; step *= 2)
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          const uint32_t next = i + step < kWords ? u[i + step] : SAME ? u[i] : 0;
          u[i] = n & (step * kEach) ? next : u[i];
        }
    }
    if constexpr (DT == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(u[e]);
    } else {
      unpack8<DT>(make_uint4(u[0], u[1], u[2], u[3]), x);
    }
  }
};

template <int DT, int W>
__device__ __forceinline__ void load_piece(const void* base, int64_t at, int K, int c, int t,
                                           float (&x)[8]) {
  Piece<DT> piece;
  piece.template load<W>(base, at, K, c, t);
  piece.template get<W>(K, c, t, x);
}

template <int DT, int W>
__device__ __forceinline__ void store_piece(void* base, int64_t at, int K, int c, int t,
                                            const float (&x)[8]) {
  const int col = row_col<W>(c, t);
  if (col + 8 <= K) {
    char* p = const_cast<char*>(element<DT>(base, at + col));
    if constexpr (DT == 0) {
      __builtin_memcpy(p, x, 32);
    } else {
      const uint4 v = pack8<DT>(x);
      __builtin_memcpy(p, &v, 16);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (col + e < K) store1<DT>(base, at + col + e, x[e]);
}

template <int W>
__device__ __forceinline__ void store_codes(int8_t* base, int64_t at, int K, int c, int t,
                                            uint2 codes) {
  const int col = row_col<W>(c, t);
  if (col + 8 <= K) {
    __builtin_memcpy(base + at + col, &codes, 8);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (col + e < K) base[at + col + e] = int8_t((e < 4 ? codes.x : codes.y) >> (8 * (e & 3)));
}

// v summed over each 16 lanes, the same bits in all of them.
__device__ __forceinline__ float row16_sum(float v) {
#define AWQ_ROR_ADD(N)                                                                         \
  v += __uint_as_float(uint32_t(                                                               \
      __builtin_amdgcn_update_dpp(0, int(__float_as_uint(v)), 0x120 + N, 0xF, 0xF, false)));
  AWQ_ROR_ADD(8) AWQ_ROR_ADD(4) AWQ_ROR_ADD(2) AWQ_ROR_ADD(1)
#undef AWQ_ROR_ADD
  return v;
}
// v summed over a wave, the same bits in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
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

// Over a row's waves. `red` holds 16 values and is used for one reduction of the
// workgroup only (or again after another barrier in between).
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (W == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  const unsigned i = threadIdx.x & 15;
  return row16_sum(i < blockDim.x / 64 ? red[i] : 0.f);
}
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* red) {
  m = wave_max(m);
  if constexpr (W == 1) return m;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  const unsigned i = threadIdx.x & 15;
  return row16_max(i < blockDim.x / 64 ? red[i] : 0u);
}

// The row's codes and step from its values.
template <int W, int V>
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
    store_codes<W>(codes, at, K, c, t, act8_codes(x[c], s));
  if (t == 0) steps[row] = s.step;
}

}  // namespace
}  // namespace awq
