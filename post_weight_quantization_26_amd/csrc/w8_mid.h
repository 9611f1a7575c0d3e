// The main loop of products with too few 256x256 tiles for 256 CUs: tiles of RA
// rows of A (output channels) x TR rows of B (tokens), both row-major, 128 bytes
// of the contraction a step (128 codes or 64 16-bit numbers).
//
//  * Four waves in 2x2, each RA/2 x TR/2 outputs as blocks of 16x16 in registers.
//  * A step's RA + TR rows of 128 bytes come by buffer_load ... lds into one of
//    3 stages, 2 steps ahead; rows past the end of A or B read as zero. 16-byte
//    chunks are XORed with (row / 2) % 8, so that 16 lanes' reads of a fragment
//    fall on distinct banks.
//  * LDS bandwidth bounds the small tiles (128x64: 72 KiB written and read a
//    step, 576 cycles, against 256 of matrix instructions). A's rows straight
//    to registers, in 16-row loads, were slower (200 tokens of 11008x4096: 32 us
//    instead of 23): such a load takes as long as 16 lines' look-ups.
//  * The grid gives each XCD its own tiles of A, with all their token tiles one
//    after the other: A's rows are read from HBM once.
#pragma once

#include "gemm_types.h"
#include "w8_common.h"

namespace awq {
namespace {

#define AWQ_LDS_PTR(p) ((__attribute__((address_space(3))) void*)(p))

constexpr int kMidStages = 3;

// One array per stage: the compiler can tell the stage being read from the one
// being filled.
template <int ROWS, int S>
__device__ __forceinline__ uint4* mid_stage() {
  __shared__ uint4 stage[ROWS * 8];
  return stage;
}

template <class V>
struct MidAcc {
  typedef floatx4 type;
};
template <>
struct MidAcc<i8x16_t> {
  typedef intx4 type;
};
__device__ __forceinline__ intx4 mid_mfma(i8x16_t a, i8x16_t b, intx4 c) {
  return mfma_16x16x64(a, b, c);
}
__device__ __forceinline__ floatx4 mid_mfma(bf16x8_t a, bf16x8_t b, floatx4 c) {
  return mfma_16x16x32(a, b, c);
}
__device__ __forceinline__ floatx4 mid_mfma(f16x8_t a, f16x8_t b, floatx4 c) {
  return mfma_16x16x32(a, b, c);
}

// s_waitcnt immediate (vmcnt in bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8):
// at most n loads in flight, no LDS read pending.
constexpr int mid_wait(int n) { return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4); }
__device__ __forceinline__ void mid_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// A tile's operands. PAIR: a wave's rows of A are RA / 4 of each of two matrices
// of equal length, so that both sums of an output lie in one lane.
struct MidTile {
  __amdgpu_buffer_rsrc_t a0, a1, b;
  int v;            // the lane's byte offset in the first 32 rows of A or B
  int copy;         // bytes of 32 rows
  int wave, past;   // past: an offset beyond every resource
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mid_rsrc(const void* base, int64_t rows,
                                                          int64_t ld) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, int(rows * ld),
                                           0x00020000);
}

// Row strides ld in bytes, below 2^23; rows_a and rows_b the valid ones of the
// tile (of a pair, of each matrix's RA / 2).
template <bool PAIR, int RA, int TR>
__device__ __forceinline__ MidTile mid_setup(const void* a0, const void* a1, int64_t rows_a,
                                             const void* b, int64_t rows_b, int64_t ld) {
  MidTile m;
  m.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  m.a0 = mid_rsrc(a0, rows_a, ld);
  m.a1 = mid_rsrc(PAIR ? a1 : a0, rows_a, ld);
  m.b = mid_rsrc(b, rows_b, ld);
  const int lane = threadIdx.x & 63;
  const int row = m.wave * 8 + (lane >> 3);         // of each copy's 32 rows
  const int chunk = (lane & 7) ^ ((row >> 1) & 7);  // a copy's first row is a multiple of 32
  m.v = row * int(ld) + chunk * 16;
  m.copy = 32 * int(ld);
  m.past = (RA > TR ? RA : TR) * int(ld);
  return m;
}

// Copies of step kt into stage S: 32 rows of A or B each, 8 of them a wave.
template <bool PAIR, int RA, int TR, int S>
__device__ __forceinline__ void mid_copy(const MidTile& m, int kt, int end) {
  const int v = m.v + (kt < end ? kt * 128 : m.past);
  uint4* s = mid_stage<RA + TR, S>();
  constexpr int H = RA / 128;   // copies of a wave's rows of one of a pair's matrices
#pragma unroll
  for (int j = 0; j < RA / 32; ++j) {
    const bool second = PAIR && (j / H) & 1;
    const int rows = PAIR ? (j / (2 * H)) * H + j % H : j;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(second ? m.a1 : m.a0,
                                             AWQ_LDS_PTR(s + (j * 32 + m.wave * 8) * 8), 16, v,
                                             rows * m.copy, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < TR / 32; ++j)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(m.b, AWQ_LDS_PTR(s + (RA + j * 32 + m.wave * 8) * 8),
                                             16, v, j * m.copy, 0, 0);
}

template <class V, int RA, int TR, int S>
__device__ __forceinline__ void mid_compute(
    const MidTile& m, typename MidAcc<V>::type (&acc)[RA / 32][TR / 32]) {
  const uint4* s = mid_stage<RA + TR, S>();
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int ra = (m.wave >> 1) * (RA / 2) + r, rb = RA + (m.wave & 1) * (TR / 2) + r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int chunk = (h * 4 + q) ^ (r >> 1);
    V a[RA / 32], b[TR / 32];
#pragma unroll
    for (int j = 0; j < TR / 32; ++j) b[j] = __builtin_bit_cast(V, s[(rb + j * 16) * 8 + chunk]);
#pragma unroll
    for (int i = 0; i < RA / 32; ++i) a[i] = __builtin_bit_cast(V, s[(ra + i * 16) * 8 + chunk]);
#pragma unroll
    for (int i = 0; i < RA / 32; ++i)
#pragma unroll
      for (int j = 0; j < TR / 32; ++j) acc[i][j] = mid_mfma(a[i], b[j], acc[i][j]);
  }
}

// One step: its copies have landed (this wave's by the wait, which leaves those of
// the step after it in flight, the others' by the barrier, which also says that
// every wave has read the stage of step kt - 1), so that stage may be filled with
// step kt + 2. N is the stage of step kt.
template <class V, bool PAIR, int RA, int TR, int N>
__device__ __forceinline__ void mid_step(const MidTile& m, int kt, int end,
                                         typename MidAcc<V>::type (&acc)[RA / 32][TR / 32]) {
  __builtin_amdgcn_s_waitcnt(mid_wait((RA + TR) / 32));
  mid_barrier();
  mid_copy<PAIR, RA, TR, (N + 2) % kMidStages>(m, kt + 2, end);
  mid_compute<V, RA, TR, N>(m, acc);
}

// Steps begin .. end - 1 into zeroed accumulators.
template <class V, bool PAIR, int RA, int TR>
__device__ __forceinline__ void mid_loop(const MidTile& m, int begin, int end,
                                         typename MidAcc<V>::type (&acc)[RA / 32][TR / 32]) {
  mid_copy<PAIR, RA, TR, 0>(m, begin, end);
  mid_copy<PAIR, RA, TR, 1>(m, begin + 1, end);
  int kt = begin;
  for (; kt + 3 <= end; kt += 3) {
    mid_step<V, PAIR, RA, TR, 0>(m, kt, end, acc);
    mid_step<V, PAIR, RA, TR, 1>(m, kt + 1, end, acc);
    mid_step<V, PAIR, RA, TR, 2>(m, kt + 2, end, acc);
  }
  if (kt < end) mid_step<V, PAIR, RA, TR, 0>(m, kt, end, acc);
  if (kt + 1 < end) mid_step<V, PAIR, RA, TR, 1>(m, kt + 1, end, acc);
  // no copy (of zeros, past the end) outlives the workgroup's LDS
  __builtin_amdgcn_s_waitcnt(mid_wait(0));
}

// Workgroup -> (A tile, token tile); false for padding.
__device__ __forceinline__ bool mid_tile_of(int bid, int tiles_a, int tiles_t, int& ta, int& tt) {
  const int xcd = bid & 7, i = bid >> 3;
  ta = (i / tiles_t) * 8 + xcd;
  tt = i % tiles_t;
  return ta < tiles_a;
}
inline int64_t mid_blocks(int64_t tiles_a, int64_t tiles_t) {
  return (tiles_a + 7) / 8 * 8 * tiles_t;
}

}  // namespace
}  // namespace awq
