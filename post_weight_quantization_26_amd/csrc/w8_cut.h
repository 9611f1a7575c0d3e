// 256x256 tiles on 256 CUs, one workgroup each: tiles past a multiple of 256
// would leave most CUs idle for a whole tile's time. These last tiles are cut
// into runs of the contraction instead; the runs' accumulators go out in
// register order (1 KiB per store) and a second launch adds them.
#pragma once

#include "w8_common.h"
#include "w8_ring.h"

namespace awq {
namespace {

// A workgroup's tile and, of a cut one, its run (slot >= 0).
struct W8Unit {
  int tt, tn, run, slot;
};

// Tile number -> (token tile, channel tile): groups of at most 6 token tiles, in each
// the channel tiles one after the other with the group's token tiles fastest.
__device__ __forceinline__ void w8_tile(int tile, int tiles_t, int tiles_n, int& tt, int& tn) {
  const int groups = (tiles_t + 5) / 6, size = (tiles_t + groups - 1) / groups;
  const int g = tile / (size * tiles_n), rest = tile - g * size * tiles_n;
  const int mine = tiles_t - g * size < size ? tiles_t - g * size : size;
  tn = rest / mine;
  tt = g * size + rest - tn * mine;
}

// Number i of n in the order that gives each XCD (consecutive workgroups go round
// them) a contiguous run of numbers: its 32 CUs work on about 5 x 6 neighbouring
// tiles, so their L2 holds what they share.
__device__ __forceinline__ int w8_of_xcd(int i, int n) {
  const int q = n / 8, rem = n % 8, x = i % 8;
  return x * q + (x < rem ? x : rem) + i / 8;
}

template <bool CUT>
__device__ __forceinline__ W8Unit w8_unit(const W8Cut& cut, int tiles_t, int tiles_n) {
  W8Unit u;
  u.run = 0;
  u.slot = -1;
  int tile;
  if constexpr (CUT) {
    const int id = int(blockIdx.x);
    if (id < cut.full) {
      tile = w8_of_xcd(id, cut.full);
    } else {
      u.slot = w8_of_xcd(id - cut.full, int(gridDim.x) - cut.full);
      tile = cut.full + u.slot / cut.runs;
      u.run = u.slot % cut.runs;
    }
  } else {
    tile = w8_of_xcd(int(blockIdx.x), int(gridDim.x));
  }
  w8_tile(tile, tiles_t, tiles_n, u.tt, u.tn);
  return u;
}

// First and last + 1 of a run's k-tiles, of `steps`.
__device__ __forceinline__ void w8_run(const W8Cut& cut, const W8Unit& u, int steps, int& k0,
                                       int& k1) {
  // at most 2^16 steps (a pair's gradient, N below 2^21) and 256 runs
  k0 = u.slot < 0 ? 0 : steps * u.run / cut.runs;
  k1 = u.slot < 0 ? steps : steps * (u.run + 1) / cut.runs;
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

// A wave's outputs, 128 tokens x COLS channels of 16 bits, through its quarter of
// the main loop's LDS: lanes hold 4 channels of a token, rows of 16 tokens; the
// stores take 16 bytes a lane and whole lines. (With 8-byte stores of 16 tokens each a
// round of 256 tiles of K = 2048 took 42 us, with these 33.) 16-byte chunks are XORed
// with the row, so that 16 lanes write or read distinct banks.
template <int COLS>
struct WaveTile {
  static constexpr int kChunks = COLS / 8;
  uint4* lds;
  __device__ __forceinline__ WaveTile(int wave)
      : lds(wave == 0 ? ring0 : wave == 1 ? ring1 : wave == 2 ? ring2 : ring3) {}
  __device__ __forceinline__ uint4* at(int t, int chunk) const {
    return lds + t * kChunks + (chunk ^ (COLS == 64 ? (t >> 1) & 7 : t & 15));
  }
  // channels n .. n + 3 (a multiple of 4) of token t
  template <bool F16>
  __device__ __forceinline__ void put(int t, int n, const float (&y)[4]) const {
    uint32_t h[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) h[v] = round16<F16>(y[v]);
    reinterpret_cast<uint2*>(at(t, n >> 3))[(n >> 2) & 1] =
        make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  }
  // To out, rows of ld elements: the first left_t tokens and left_n channels.
  __device__ __forceinline__ void store(uint16_t* out, uint32_t ld, int left_t, int left_n) const {
    const int lane = threadIdx.x & 63, n = lane % kChunks * 8;
#pragma unroll
    for (int i = 0; i < 128 * kChunks / 64; ++i) {
      const int t = i * (64 / kChunks) + lane / kChunks;
      const uint4 v = *at(t, lane % kChunks);
      if (t >= left_t || n >= left_n) continue;
      uint16_t* o = out + (uint32_t(t) * ld + uint32_t(n));
      if (n + 8 <= left_n) {
        __builtin_memcpy(o, &v, 16);   // rows of any length: at any element's address
        continue;
      }
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (n + e < left_n) o[e] = uint16_t(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]);
    }
  }
};

}  // namespace
}  // namespace awq
