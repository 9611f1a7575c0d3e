// 256x256 tiles on 256 CUs, one workgroup each: tiles past a multiple of 256
// would leave most CUs idle for a whole tile's time. These last tiles are cut
// into runs of the contraction instead; the runs' accumulators go out in
// register order (1 KiB per store) and a second launch adds them.
#pragma once

#include "gemm_core.h"
#include "w8_common.h"

namespace awq {
namespace {

// The main loop's context with everything that the compiler has to know to be
// uniform said so: else every copy is a loop over the lanes' resources (4096
// tokens of 4096x11008: 165 instead of 150 us).
template <class T>
__device__ __forceinline__ const T* uniform(const T* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(u)),
                 hi = __builtin_amdgcn_readfirstlane(uint32_t(u >> 32));
  return reinterpret_cast<const T*>(uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ void w8_setup(GemmCtx64& c, const uint16_t* A, int64_t rows_a,
                                         const uint16_t* B, int64_t rows_b, int64_t ld,
                                         int64_t k) {
  gemm_setup64(c, uniform(A), __builtin_amdgcn_readfirstlane(int(rows_a)), ld, uniform(B),
               __builtin_amdgcn_readfirstlane(int(rows_b)), ld, k, false);
  c.KT = __builtin_amdgcn_readfirstlane(c.KT);
}

// A workgroup's tile and, of a cut one, its run (slot >= 0).
struct W8Unit {
  int tt, tn, run, slot;
};

// Token tile fastest; XCD i takes a contiguous run of the whole tiles, and of the
// (tile, run) units behind them. False for padding.
template <bool CUT>
__device__ __forceinline__ bool w8_unit(const W8Cut& cut, int tiles_t, int tiles_n, W8Unit& u) {
  u.run = 0;
  u.slot = -1;
  if constexpr (CUT) {
    int tile;
    const int id = int(blockIdx.x);
    if (id < cut.full) {
      tile = (id % 8) * (cut.full / 8) + id / 8;
    } else {
      const int v = id - cut.full, units = int(gridDim.x) - cut.full, q = units / 8,
                rem = units % 8, x = v % 8;
      u.slot = x * q + (x < rem ? x : rem) + v / 8;
      tile = cut.full + u.slot / cut.runs;
      u.run = u.slot % cut.runs;
    }
    u.tt = tile % tiles_t;
    u.tn = tile / tiles_t;
  } else {
    if (!tile_of(blockIdx.x, tiles_t, tiles_n, u.tt, u.tn)) return false;
  }
  return true;
}

// First and last + 1 of a run's elements among `steps` 64-wide k-tiles.
__device__ __forceinline__ void w8_run(const W8Cut& cut, const W8Unit& u, int steps, int64_t& k0,
                                       int64_t& k1) {
  k0 = u.slot < 0 ? 0 : int64_t(steps) * u.run / cut.runs * BK64;
  k1 = u.slot < 0 ? int64_t(steps) * BK64 : int64_t(steps) * (u.run + 1) / cut.runs * BK64;
}

// Keeps an accumulator in its AGPRs up to this use: with two ways out of a kernel
// the compiler copied all of them to vector registers ahead, and spilled.
__device__ __forceinline__ floatx4 from_agpr(floatx4& acc) {
  asm volatile("" : "+a"(acc));
  return acc;
}

__device__ __forceinline__ void w8_store_run(const W8Cut& cut, const W8Unit& u, int wave,
                                             floatx4 (&acc)[8][8]) {
  floatx4* out = reinterpret_cast<floatx4*>(cut.part) + (int64_t(u.slot) * 4 + wave) * 4096 +
                 (threadIdx.x & 63);
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) out[(i * 8 + j) * 64] = from_agpr(acc[i][j]);
}

// The sum over the runs of cut tile `tile`, block (i, j) of a wave, in the runs'
// order. V: floatx4 or intx4.
template <class V>
__device__ __forceinline__ V w8_sum_runs(const W8Cut& cut, int tile, int wave, int i, int j) {
  const V* src = reinterpret_cast<const V*>(cut.part) +
                 (int64_t(tile) * cut.runs * 4 + wave) * 4096 + (i * 8 + j) * 64 +
                 (threadIdx.x & 63);
  V s = src[0];
#pragma unroll 4
  for (int r = 1; r < cut.runs; ++r) s += src[int64_t(r) * 4 * 4096];
  return s;
}

}  // namespace
}  // namespace awq
